// attention_decode.cu -- attention of one new token per sequence over a paged key-value cache (moe_attention_decode,
// include/moe.h).
//
//   out_h = sum_t p_t v_t / sum_t p_t,   p_t = 2^(s_t - m),  s_t = scale * log2(e) * (q_h . k_t)
//
// The cache is read once and nothing else counts: 4 * head_dim bytes a token and key head, for 4 * head_dim flops a
// query head.  So this is a stream, like the weight stream of linear.cu: a CTA per SM with a ring of up to 200 KB of
// shared memory, and two teams in it that share the ring's slots and nothing else: two warps that load tiles of 64 or 128
// tokens (keys, and values, of one key head, by TMA through the page table; a stretch's queries ahead of its first tile,
// 222 -> 218 us for the 88 sequences below) and four that take 16 tokens of each 64.  Two
// warp-level MMAs per 16 x 16 values of a tile do the work of all query heads that share the key head, eight at a time:
//   S^T[16 tokens, 8 heads] = K Q^T,    O^T[16 values, 8 heads] += V^T P^T    (BF16: P as two numbers, two MMAs)
// With tokens as the rows of the first product and values as the rows of the second, keys come out of shared memory as
// they lie there (16 bytes a lane, which pair with the same 16 bytes of q), values by one byte permutation per pair of
// tokens, and P moves from one to the other by a transposition of 8 x 8 (movmatrix).  The tiles carry TMA's 128-byte
// (8-bit heads of 64: 64-byte) swizzle, so that neither read meets a bank twice.
//
// The work of all sequences and key heads, tile by tile, is one long list that the workers (the teams of all CTAs) share
// evenly whatever the lengths (which only the device knows): worker w takes the places [w * share, (w + 1) * share).  What
// it finishes alone it writes; of a sequence and head that other workers have a part of it leaves the running maximum, sum
// and vector in the workspace, and a second kernel joins the parts in their order.  (Both teams on one list, each taking
// every other tile, left the SM idle while a sequence's end was written and the next one's start loaded: 88 sequences of
// 1 to 256 tokens 24.8 us for 18.9, the MXFP8 case below 267 for 249.)
//
// MXFP8 caches (half the bytes): E4M3 values become FP16 exactly.  A block's power of two is applied to the FP32 sums
// of its 32 values (keys), or to P (values), relative to a power that the vector's block is kept in; tokens whose powers
// lie too far from it for FP16 are taken one by one in FP32.  That power is a stretch's own (kept from one to the next it
// let a sequence's largest values reach the sums of others; the 176 sequences below, with v of 2^6 from head to head, then
// took 645 us for 247).  With one token in 64 that lies 2^5 above the rest most tokens of every fourth warp go one by one,
// and the others wait for it: 1002 us.
//
// Measured (device time among other calls; 64 query heads on 8 key heads of 128 if not said otherwise): one sequence of
// 131072 tokens 85 us (537 MB, 0.93 of a plain copy's rate; 80 without the join); 88 sequences of 0 to 8192 (56 on 8)
// 218 us (1.49 GB, 1.00); 176 of 1 to 8192 in MXFP8 246 us (1.53 GB, 0.92); 15 of 1 to 4096, 32 heads of 64 unshared,
// pages of 16 tokens, 44 us (245 MB, 0.82: 2 KB a copy); one of 1000 tokens (56 on 8) 8.1 us, a chain of latencies:
// lengths, page numbers, tiles, parts, join.  Up to 16 query heads to a key head take two products of eight: 88 sequences
// of 0 to 8192, 64 heads on 4, 133 us (0.82) in BF16 and 103 (0.55) in MXFP8, 96 on 8 248 (0.88) and 189 (0.60); heads of
// 128 then spill 32 and 68 bytes a thread.  Beyond 16 the cache is read once for each 16: 32 sequences of 4096, 40 heads on
// 1, 41.6 us (0.24) and 36.7 (0.14).
#include <math.h>
#include <stdio.h>

#include "attention_internal.cuh"
#include "gemm_common.cuh"
#include "mx_encode.cuh"
#include "overlap.cuh"

namespace moe {

namespace {

using namespace gemm;

constexpr int TEAM = 4;              // warps that share a tile, 16 tokens of each 64
constexpr int TEAMS = 2;             // of a CTA, each with tiles of its own
constexpr int MAX_STAGES = 16;
// Tiles of a worker at least: shared 1 (one sequence of 1000 tokens 7.9 us, with 2 8.5), whole 2 (16 of 1 to 256 tokens 8.3
// us, with 1 9.0).
constexpr int MIN_SHARE = 1, MIN_WHOLE = 2;

// A unit that starts with a worker (as its first stretch or its last: part 0 or 1) and ends with worker `last`; of the
// workers between it is the first stretch.  heads == 0: there is none.
struct alignas(16) Split {
    int b, head, heads_part, last;  // heads_part: heads * 2 + part
};

struct DecodeArgs {
    const uint16_t *q;
    long long q_ld;
    const int32_t *table;
    int max_pages;
    const int32_t *lens;
    long long cap;                   // tokens that a row of the table holds
    int B, heads, kv, group;         // group: query heads of a key head
    int chunks, units;               // chunks of up to 8 NT heads of a group; units = kv * chunks
    int n_pages, page_log2;
    const uint8_t *ks, *vs;
    float scale;                     // times log2(e)
    uint16_t *out;
    long long out_ld;
    float *part_o, *part_ml;         // parts: [2 * workers][8 NT][D], [2 * workers][8 NT][2]
    Split *splits;                   // [workers]: what starts with one and goes on with the next
    int ctas, workers;               // the workers are the CTAs' teams, all first ones first
    bool whole;                      // a unit is its first place's worker's alone
    int *err;
};

template <int D, int NT, bool MX> struct Geo {
    static constexpr int WARPS = TEAM * TEAMS;       // that compute
    static constexpr int LOADERS = 2 * TEAMS;        // one for a team's keys, one for its values
    static constexpr int THREADS = (WARPS + LOADERS) * 32;
    static constexpr int ROW_B = D * (MX ? 1 : 2);
    // tokens of a tile: 64 in BF16, 128 where they have half the bytes or fewer (waiting, arming and asking for a tile
    // cost about 180 instructions per warp and tile, as many as 16 tokens' keys)
    static constexpr int TILE = ROW_B >= 256 ? 64 : 128;
    static constexpr int TILE_B = TILE * ROW_B;
    static constexpr int SC_B = MX ? TILE * D / 32 : 0;
    // what starting and ending a sequence and head costs, in tiles (0.7 us; a tile's bytes take 0.73 us per 32 KB)
    static constexpr int START = TILE_B >= 16384 ? 1 : 2;
    static constexpr int MERGE_B = TEAMS * 2 * NT * 8 * D * 4;         // two partial vectors of a team's heads
    static constexpr int Q_B = NT * 8 * D * 2;                         // the queries of a stretch
    static constexpr int ML_B = WARPS * NT * 8 * 2 * 4;
    static constexpr int FIT = (224 * 1024 - MERGE_B - 2 * ML_B - 2 * TEAMS * Q_B) / (2 * (TILE_B + SC_B));
    // a multiple of the teams: a slot then is one team's, which so sees every phase of its barriers
    static constexpr int STAGES = (FIT < MAX_STAGES ? FIT : MAX_STAGES) / TEAMS * TEAMS;
    static constexpr int SC_OFF = STAGES * 2 * TILE_B;
    static constexpr int MERGE_OFF = SC_OFF + STAGES * 2 * SC_B;
    static constexpr int ML_OFF = MERGE_OFF + MERGE_B;                 // [2][TEAMS][TEAM][8 NT][2]
    static constexpr int Q_OFF = ML_OFF + 2 * ML_B;                    // [TEAMS][2]
    static constexpr int BAR_OFF = Q_OFF + 2 * TEAMS * Q_B;
    static constexpr int BAD_OFF = BAR_OFF + (2 * MAX_STAGES + 4 * TEAMS) * 8;       // a stage holds a page outside the cache
    static constexpr int SMEM = BAD_OFF + MAX_STAGES * 4 + 1024;       // + alignment slack
    static_assert(SMEM <= 226 * 1024, "shared memory");
    static_assert(TILE_B % 1024 == 0 && SC_OFF % 16 == 0 && SC_B % 16 == 0 && Q_OFF % 16 == 0 && BAR_OFF % 8 == 0,
                  "alignment");
};

// Tiles of a sequence of n tokens: 0 for an empty one and for a length that the table cannot hold.
template <class G> __device__ __forceinline__ int tiles_of(const DecodeArgs &a, int n)
{
    return n > 0 && n <= a.cap ? (n + G::TILE - 1) / G::TILE : 0;
}

// The places of the list that a worker takes, of `total` in all.  A unit (a key head of a sequence, or a chunk of its
// query heads) has START places for its beginning and end before one place per tile.
template <class G> __device__ __forceinline__ long long share_of(const DecodeArgs &a, long long total)
{
    const long long s = (total + a.workers - 1) / a.workers;
    const int least = G::START + (a.whole ? MIN_WHOLE : MIN_SHARE);
    return s < least ? least : s;
}

template <class G> __device__ __forceinline__ int places_of(const DecodeArgs &a, int b)
{
    const int nt = tiles_of<G>(a, __ldcg(a.lens + b));
    return nt ? nt + G::START : 0;
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <bool F16>
__device__ __forceinline__ void mma16816(float c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    if (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// a and b, 0 or more, as two BF16 numbers each: what the first, their upper half, leaves goes into the second, which is
// above 0 wherever the first is (a zero or a negative number times an infinite value would make NaN of it).  Their sum is
// off by 2^-15 of a or b.
__device__ __forceinline__ void bf16_in_two(float a, float b, uint32_t &first, uint32_t &second)
{
    constexpr float LEAST = 1.f / (1 << 17);
    first = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
    second = bf16_pair(fmaxf(a - __uint_as_float(__float_as_uint(a) & 0xFFFF0000u), a * LEAST),
                       fmaxf(b - __uint_as_float(__float_as_uint(b) & 0xFFFF0000u), b * LEAST));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ uint32_t f16_pair(float a, float b)
{
    const __half2 p = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&p);
}

__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)v));
    return h;
}

// 2^(byte - 127), NaN for 255
__device__ __forceinline__ float e8m0(uint32_t byte)
{
    return byte == 255 ? __int_as_float(0x7FC00000) : __int_as_float(byte ? byte << 23 : 0x400000);
}

__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

__device__ __forceinline__ uint2 lds64(uint32_t a)
{
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}

__device__ __forceinline__ uint32_t lds32(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}

__device__ __forceinline__ uint32_t lds16(uint32_t a)
{
    uint16_t v;
    asm volatile("ld.shared.b16 %0, [%1];" : "=h"(v) : "r"(a));
    return v;
}

__device__ __forceinline__ void tma_4d(void *dst, const CUtensorMap *map, int x, int y, int z, int w, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
        "%5}], [%6];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
        : "memory");
}

// What one warp of those that compute holds of a sequence and key head: per lane (g, q) = (lane / 4, lane % 4) the
// vector's values of heads 2q and 2q + 1, their maximum (of log2 scores) and its own part of their sum.
template <int D, int NT> struct State {
    float o[D / 16][NT][4];
    float m[NT][2], l[NT][2];
};

// ---------------------------------------------------------------- BF16

// q (in shared memory) as the B operand: lane (g, q) has of head g the 16-byte pieces 8 h + 2q and 8 h + 2q + 1 of each
// 64 values h
template <int D, int NT>
__device__ __forceinline__ void load_q(uint32_t q, int heads, int g, int qd, uint32_t (&qf)[NT][D / 8])
{
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            uint4 u = make_uint4(0, 0, 0, 0);
            if (8 * nt + g < heads)
                u = lds128(q + (8 * nt + g) * (D * 2) + (8 * (c / 2) + 2 * qd + (c & 1)) * 16);
            qf[nt][4 * c] = u.x, qf[nt][4 * c + 1] = u.y, qf[nt][4 * c + 2] = u.z, qf[nt][4 * c + 3] = u.w;
        }
}

// Scores' maximum over the 16 tokens, per head; s turns into scaled scores, -inf past the sequence
template <int NT>
__device__ __forceinline__ void tile_max(float (&s)[NT][4], const float (&mul)[NT][2], bool in0, bool in1,
                                         float (&mt)[NT][2])
{
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        s[nt][0] = in0 ? s[nt][0] * mul[nt][0] : -INFINITY;
        s[nt][1] = in0 ? s[nt][1] * mul[nt][1] : -INFINITY;
        s[nt][2] = in1 ? s[nt][2] * mul[nt][0] : -INFINITY;
        s[nt][3] = in1 ? s[nt][3] * mul[nt][1] : -INFINITY;
        mt[nt][0] = fmaxf(s[nt][0], s[nt][2]);
        mt[nt][1] = fmaxf(s[nt][1], s[nt][3]);
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            mt[nt][0] = fmaxf(mt[nt][0], __shfl_xor_sync(0xffffffffu, mt[nt][0], o));
            mt[nt][1] = fmaxf(mt[nt][1], __shfl_xor_sync(0xffffffffu, mt[nt][1], o));
        }
}

__device__ __forceinline__ float finite_base(float m) { return m == -INFINITY ? 0.f : m; }

// The running maxima with those of 16 more tokens
template <int D, int NT> __device__ __forceinline__ void grow(State<D, NT> &st, const float (&mt)[NT][2])
{
    bool grown = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
        grown |= mt[nt][0] > st.m[nt][0] || mt[nt][1] > st.m[nt][1];
    if (!__any_sync(0xffffffffu, grown))
        return;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float m = fmaxf(st.m[nt][h], mt[nt][h]), f = ex2(st.m[nt][h] - finite_base(m));
            st.m[nt][h] = m;
            st.l[nt][h] *= f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                st.o[i][nt][h] *= f;
                st.o[i][nt][2 + h] *= f;
            }
        }
    }
}

// 16 tokens of a BF16 tile.  kb, vb: shared addresses of the warp's block of rows (of `rows` rows), r0 its first row
// there; n of the 16 tokens belong to the sequence.
template <int D, int NT>
__device__ __forceinline__ void tile_bf16(State<D, NT> &st, const uint32_t (&qf)[NT][D / 8], uint32_t kb, uint32_t vb,
                                          int rows, int r0, int n, const float (&mul)[NT][2], int g, int qd)
{
    float sa[NT][4], sb[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            sa[nt][i] = sb[nt][i] = 0.f;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
        const uint32_t at = kb + (c / 2) * rows * 128 + (r0 + g) * 128 + (((2 * qd + (c & 1)) ^ g) << 4);
        const uint4 k0 = lds128(at), k1 = lds128(at + 8 * 128);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            mma16816<false>(sa[nt], k0.x, k1.x, k0.y, k1.y, qf[nt][4 * c], qf[nt][4 * c + 1]);
            mma16816<false>(sb[nt], k0.z, k1.z, k0.w, k1.w, qf[nt][4 * c + 2], qf[nt][4 * c + 3]);
        }
    }
    float mt[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            sa[nt][i] += sb[nt][i];
    tile_max<NT>(sa, mul, g < n, g + 8 < n, mt);
    grow<D, NT>(st, mt);
    uint32_t pf[NT][2], rest[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const float b0 = finite_base(st.m[nt][0]), b1 = finite_base(st.m[nt][1]);
        const float p0 = ex2(sa[nt][0] - b0), p1 = ex2(sa[nt][1] - b1);
        const float p2 = ex2(sa[nt][2] - b0), p3 = ex2(sa[nt][3] - b1);
        st.l[nt][0] += p0 + p2;
        st.l[nt][1] += p1 + p3;
        // v is BF16, and an MMA's operands share a type: P goes in as two BF16 numbers, in a product each.  (The tensor pipe
        // has room: it stood at 8 % with one product, which put outputs off by up to another BF16 rounding.)
        uint32_t first[2], second[2];
        bf16_in_two(p0, p1, first[0], second[0]);
        bf16_in_two(p2, p3, first[1], second[1]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            pf[nt][i] = transpose8x8(first[i]);
            rest[nt][i] = transpose8x8(second[i]);
        }
    }
#pragma unroll
    for (int h = 0; h < D / 64; ++h) {
        uint4 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 2 * qd + (i & 1) + 8 * (i >> 1);
            w[i] = lds128(vb + h * rows * 128 + (r0 + t) * 128 + ((g ^ (t & 7)) << 4));
        }
        if (n < 16) {
#pragma unroll
            for (int i = 0; i < 4; ++i)  // what lies past the end may be anything: 0 * inf is not 0
                if (2 * qd + (i & 1) + 8 * (i >> 1) >= n)
                    w[i] = make_uint4(0, 0, 0, 0);
        }
        const uint32_t w0[4] = {w[0].x, w[0].y, w[0].z, w[0].w}, w1[4] = {w[1].x, w[1].y, w[1].z, w[1].w};
        const uint32_t w2[4] = {w[2].x, w[2].y, w[2].z, w[2].w}, w3[4] = {w[3].x, w[3].y, w[3].z, w[3].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t a0 = __byte_perm(w0[i], w1[i], 0x5410), a1 = __byte_perm(w0[i], w1[i], 0x7632);
            const uint32_t a2 = __byte_perm(w2[i], w3[i], 0x5410), a3 = __byte_perm(w2[i], w3[i], 0x7632);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                mma16816<false>(st.o[4 * h + i][nt], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
                mma16816<false>(st.o[4 * h + i][nt], a0, a1, a2, a3, rest[nt][0], rest[nt][1]);
            }
        }
    }
}

// ---------------------------------------------------------------- MXFP8

// q in FP16 with a power of two per head (the largest |q| lands in [2^14, 2^15)): lane (g, q) has of head g the values
// 32 b + 8 q .. + 7 of each block b.  e: the powers of heads 2q and 2q + 1.
template <int D, int NT>
__device__ __forceinline__ void load_q_f16(float scale, uint32_t q, int heads, int g, int qd, uint32_t (&qf)[NT][D / 8],
                                           float (&mul)[NT][2])
{
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        uint32_t w[D / 8];
        float m = 0.f;  // (NaN is left out and stays NaN in FP16)
#pragma unroll
        for (int b = 0; b < D / 32; ++b) {
            uint4 u = make_uint4(0, 0, 0, 0);
            if (8 * nt + g < heads)
                u = lds128(q + (8 * nt + g) * (D * 2) + (4 * b + qd) * 16);
            w[4 * b] = u.x, w[4 * b + 1] = u.y, w[4 * b + 2] = u.z, w[4 * b + 3] = u.w;
        }
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
            m = fmaxf(m, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xFFFF0000u))));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const int e = max((int)(__float_as_uint(m) >> 23) - 141, -126);
        const float by = __int_as_float((127 - e) << 23);
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
            qf[nt][i] = f16_pair(__uint_as_float(w[i] << 16) * by, __uint_as_float(w[i] & 0xFFFF0000u) * by);
        mul[nt][0] = scale * __int_as_float((127 + __shfl_sync(0xffffffffu, e, 8 * qd)) << 23);
        mul[nt][1] = scale * __int_as_float((127 + __shfl_sync(0xffffffffu, e, 8 * qd + 4)) << 23);
    }
}

// {2^(b0 - 127), 2^(b1 - 127)} of two E8M0 bytes as floats, NaN for 255
__device__ __forceinline__ float2 e8m0x2(uint32_t bytes)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(r) : "h"((uint16_t)bytes));
    return make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xFFFF0000u));
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The scales of tokens t and t + 1 (t even)
template <int D> __device__ __forceinline__ uint2 scales_of_two(uint32_t base, int t)
{
    if (D == 128)
        return lds64(base + t * 4);
    const uint32_t v = lds32(base + t * 2);
    return make_uint2(v & 0xFFFFu, v >> 16);
}

// The powers of two in use for the blocks of values, as E8M0 bytes: a state's vector is relative to them.  They are a
// stretch's own: the largest of its first 16 tokens', and later of others that lie too far from them; but 2^53 at most, so
// that the power of an infinity (2^120 from the cache's writer) does not put the other tokens' products below FP32's
// range.  (A product of P, up to 2^12, and a value relative to 2^53 is below 2^(12 + 127 - 53 + 9): sums have 2^33 to spare.)
constexpr int MOST_POWER = 180;

struct Powers {
    uint32_t bytes;
    bool narrow;  // none below 16
    bool fresh;   // nothing is relative to them yet
};

// The lane's token's scale bytes of values, 0 past the end
template <int D> __device__ __forceinline__ uint32_t value_scales(uint32_t vsb, int n, int lane)
{
    return lane >= n ? 0u : D == 128 ? lds32(vsb + lane * 4) : lds16(vsb + lane * 2);
}

// The largest power of block b among the lanes' tokens' (that of NaN counts for none: its products are NaN anyway)
__device__ __forceinline__ uint32_t largest_power(uint32_t mine, int b)
{
    const uint32_t power = (mine >> (8 * b)) & 255;
    return min((uint32_t)MOST_POWER, __reduce_max_sync(0xffffffffu, power == 255 ? 0u : power));
}

// The first tokens' powers
template <int D> __device__ __forceinline__ void start_powers(Powers &ref, uint32_t vsb, int n, int lane)
{
    const uint32_t mine = value_scales<D>(vsb, n, lane);
    ref = {0, true, false};
#pragma unroll
    for (int b = 0; b < D / 32; ++b) {
        const uint32_t top = largest_power(mine, b);
        ref.bytes |= top << (8 * b);
        ref.narrow = ref.narrow && top >= 16;
    }
}

// 16 tokens' values where their blocks' powers lie far from those in use: a token at a time in FP32.
template <int D, int NT>
__device__ __forceinline__ void values_apart(State<D, NT> &st, const float (&p)[NT][4], uint32_t vb, uint32_t vsb, int r0, int n,
                                          Powers &ref, int lane)
{
    constexpr int NB = D / 32;
    const int g = lane >> 2, qd = lane & 3;
    const uint32_t mine = value_scales<D>(vsb, n, lane);
    uint32_t now = 0;
    ref.narrow = true;
#pragma unroll
    for (int b = 0; b < NB; ++b) {  // what is in use grows to the largest of these tokens', and the vector follows
        const uint32_t was = (ref.bytes >> (8 * b)) & 255, top = max(was, largest_power(mine, b));
        now |= top << (8 * b);
        ref.narrow = ref.narrow && top >= 16;
        const bool nan = __any_sync(0xffffffffu, ((mine >> (8 * b)) & 255) == 255);  // (and so all of the block)
        const float f = nan ? __int_as_float(0x7FC00000) : ex2((float)((int)was - (int)top));
#pragma unroll
        for (int i = 2 * b; i < 2 * b + 2; ++i)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    st.o[i][nt][c] *= f;
    }
    ref.bytes = now;
#pragma unroll 1
    for (int t = 0; t < n; ++t) {
        const uint32_t scales = D == 128 ? lds32(vsb + t * 4) : lds16(vsb + t * 2);
        float pt[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                pt[nt][h] = __shfl_sync(0xffffffffu, t < 8 ? p[nt][h] : p[nt][2 + h], 4 * (t & 7) + qd);
        const int r = r0 + t;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const float f = ex2((float)((int)((scales >> (8 * b)) & 255) - (int)((now >> (8 * b)) & 255)));
            const int byte = 32 * b + 4 * g;
            const uint32_t w = lds32(vb + (D == 128 ? r * 128 + (byte ^ ((r & 7) << 4))
                                                    : r * 64 + (byte ^ (((r >> 1) & 3) << 4))));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t x = e4m3x2_to_f16x2(j ? w >> 16 : w);
                const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&x));
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        st.o[2 * b + j][nt][h] = fmaf(pt[nt][h] * f, v.x, st.o[2 * b + j][nt][h]);
                        st.o[2 * b + j][nt][2 + h] = fmaf(pt[nt][h] * f, v.y, st.o[2 * b + j][nt][2 + h]);
                    }
            }
        }
    }
}

// log2 of the largest P, and so of what sums and vectors of MXFP8 tiles are scaled by: times 2^3 (below) it is 2^15
constexpr float RAISED = 12.f;

// 16 tokens of an MXFP8 tile.  kb, vb: shared addresses of the warp's 16 rows (a multiple of 16 into a tile that starts
// on 1024 bytes); ksb, vsb: their scales.
template <int D, int NT>
__device__ __forceinline__ void tile_mx(State<D, NT> &st, const uint32_t (&qf)[NT][D / 8], uint32_t kb, uint32_t vb,
                                        uint32_t ksb, uint32_t vsb, int n, const float (&mul)[NT][2], Powers &ref, int lane)
{
    constexpr int NB = D / 32, ROW = D;
    constexpr uint32_t SCALES = D == 128 ? 0xFFFFFFFFu : 0xFFFFu;
    const int g = lane >> 2, qd = lane & 3;
    float s[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            s[nt][i] = 0.f;
    const uint32_t k0s = D == 128 ? lds32(ksb + g * 4) : lds16(ksb + g * 2);
    const uint32_t k1s = D == 128 ? lds32(ksb + g * 4 + 32) : lds16(ksb + g * 2 + 16);
    // 8 bytes of row g, and of row g + 8: the swizzle is an exclusive or on bits 4 .. 6 of a row's byte, as is the step
    // from block to block
    const uint32_t ka = kb + g * ROW + ((8 * qd) ^ (D == 128 ? g << 4 : ((g >> 1) & 3) << 4));
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const uint2 k0 = lds64(ka ^ (32 * b)), k1 = lds64((ka ^ (32 * b)) + 8 * ROW);
        const uint32_t x0 = e4m3x2_to_f16x2(k0.x), x1 = e4m3x2_to_f16x2(k0.x >> 16);
        const uint32_t x2 = e4m3x2_to_f16x2(k0.y), x3 = e4m3x2_to_f16x2(k0.y >> 16);
        const uint32_t y0 = e4m3x2_to_f16x2(k1.x), y1 = e4m3x2_to_f16x2(k1.x >> 16);
        const uint32_t y2 = e4m3x2_to_f16x2(k1.y), y3 = e4m3x2_to_f16x2(k1.y >> 16);
        const float2 e0 = e8m0x2(k0s >> (16 * (b / 2))), e1 = e8m0x2(k1s >> (16 * (b / 2)));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float c[4] = {0.f, 0.f, 0.f, 0.f};
            mma16816<true>(c, x0, y0, x1, y1, qf[nt][4 * b], qf[nt][4 * b + 1]);
            mma16816<true>(c, x2, y2, x3, y3, qf[nt][4 * b + 2], qf[nt][4 * b + 3]);
            s[nt][0] = fmaf(c[0], b & 1 ? e0.y : e0.x, s[nt][0]);
            s[nt][1] = fmaf(c[1], b & 1 ? e0.y : e0.x, s[nt][1]);
            s[nt][2] = fmaf(c[2], b & 1 ? e1.y : e1.x, s[nt][2]);
            s[nt][3] = fmaf(c[3], b & 1 ? e1.y : e1.x, s[nt][3]);
        }
    }
    float mt[NT][2];
    tile_max<NT>(s, mul, g < n, g + 8 < n, mt);
    grow<D, NT>(st, mt);
    float p[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const float b0 = finite_base(st.m[nt][0]), b1 = finite_base(st.m[nt][1]);
        p[nt][0] = ex2(s[nt][0] - b0 + RAISED), p[nt][1] = ex2(s[nt][1] - b1 + RAISED);
        p[nt][2] = ex2(s[nt][2] - b0 + RAISED), p[nt][3] = ex2(s[nt][3] - b1 + RAISED);
        st.l[nt][0] += p[nt][0] + p[nt][2];
        st.l[nt][1] += p[nt][1] + p[nt][3];
    }
    // P, at most 2^RAISED, rounds to FP16 and takes, per block, what the token's power is away from the one in use: 2^-4 to
    // 2^3, exact but for numbers below FP16's normal range.  A probability so is off by 2^-11 of itself or 2^-37 of the
    // largest, times 2^4 at most in units of the token's values.  (With P at most 1 and 2^-25, 131,072 tokens that lay 2^-23
    // below a maximum lost most of their share.)  The usual case is that all 16 tokens fit in all blocks: then no byte
    // of `away`, power - (ref - 4), borrows from the next or has more than three bits (ref lies in 16 .. MOST_POWER, so
    // that a byte which borrows shows it, and that of NaN does not fit).
    const uint2 v01 = scales_of_two<D>(vsb, 2 * qd), v89 = scales_of_two<D>(vsb, 2 * qd + 8);
    uint32_t away[4];
    auto fit = [&] {
        away[0] = v01.x, away[1] = v01.y, away[2] = v89.x, away[3] = v89.y;
        if (n < 16) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                away[i] = 2 * qd + (i & 1) + 8 * (i >> 1) < n ? away[i] : ref.bytes;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            away[i] -= ref.bytes - (0x04040404u & SCALES);
        return __all_sync(0xffffffffu, ref.narrow && ((away[0] | away[1] | away[2] | away[3]) & 0xF8F8F8F8u) == 0) != 0;
    };
    if (!fit()) {
        const bool fresh = ref.fresh;
        if (fresh)
            start_powers<D>(ref, vsb, n, lane);
        if (!fresh || !fit()) {
            values_apart<D, NT>(st, p, vb, vsb, 0, n, ref, lane);
            return;
        }
    }
    uint32_t pt[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        pt[nt][0] = transpose8x8(f16_pair(p[nt][0], p[nt][1]));
        pt[nt][1] = transpose8x8(f16_pair(p[nt][2], p[nt][3]));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        away[i] = (away[i] << 2) + 0x2C2C2C2Cu;  // 15 + power - ref, where FP16 has its exponent in the upper byte
    // 4 bytes of row 2 q, and of the rows 1, 8 and 9 on: the next row flips bit 4 of the swizzle (with 64-byte rows it
    // has the same one)
    const uint32_t va = vb + 2 * qd * ROW + ((4 * g) ^ (D == 128 ? (2 * qd) << 4 : qd << 4));
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const uint32_t v0 = va ^ (32 * b), v1 = D == 128 ? (v0 + ROW) ^ 16 : v0 + ROW;
        uint32_t w[4] = {lds32(v0), lds32(v1), lds32(v0 + 8 * ROW), lds32(v1 + 8 * ROW)};
        if (n < 16) {
#pragma unroll
            for (int i = 0; i < 4; ++i)  // what lies past the end may be NaN: 0 * NaN is not 0
                w[i] = 2 * qd + (i & 1) + 8 * (i >> 1) < n ? w[i] : 0;
        }
        const uint32_t f01 = __byte_perm(away[0], away[1], b * 0x1111 + 0x4400) & 0xFF00FF00u;
        const uint32_t f89 = __byte_perm(away[2], away[3], b * 0x1111 + 0x4400) & 0xFF00FF00u;
        uint32_t pf[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            pf[nt][0] = mul_f16x2(pt[nt][0], f01);
            pf[nt][1] = mul_f16x2(pt[nt][1], f89);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t lo = __byte_perm(w[0], w[1], j ? 0x7362 : 0x5140);
            const uint32_t hi = __byte_perm(w[2], w[3], j ? 0x7362 : 0x5140);
            const uint32_t a0 = e4m3x2_to_f16x2(lo), a1 = e4m3x2_to_f16x2(lo >> 16);
            const uint32_t a2 = e4m3x2_to_f16x2(hi), a3 = e4m3x2_to_f16x2(hi >> 16);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                mma16816<true>(st.o[2 * b + j][nt], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
        }
    }
}

// ---------------------------------------------------------------- kernel

// A stretch of the list: tiles t0 .. t1 - 1 of unit u of sequence b, which has `len` tokens in `nt` tiles; the unit's
// places start at v.  ahead: the length of the sequence after it, asked for early.
struct Stretch {
    long long v;
    int b, len, nt, u, t0, t1, ahead;
};

template <class G> __device__ __forceinline__ void enter_sequence(const DecodeArgs &a, Stretch &p, int len)
{
    p.len = len;
    p.nt = tiles_of<G>(a, len);
    p.ahead = p.b + 1 < a.B ? __ldcg(a.lens + p.b + 1) : 0;
}

template <class G> __device__ __forceinline__ void cut(const DecodeArgs &a, Stretch &p, long long end)
{
    p.t1 = a.whole ? p.nt : (int)max(0ll, min((long long)p.nt, end - p.v - G::START));
}

// The next stretch of a worker whose places end at `end`; false where there is none.
template <class G> __device__ __forceinline__ bool advance(const DecodeArgs &a, Stretch &p, long long end)
{
    p.v += p.nt + G::START;
    if (p.t1 < p.nt || p.v + (a.whole ? 0 : G::START) >= end)
        return false;
    if (++p.u == a.units) {
        p.u = 0;
        do {
            ++p.b;
            enter_sequence<G>(a, p, p.ahead);
        } while (p.nt == 0 && p.b < a.B);
    }
    p.t0 = 0;
    cut<G>(a, p, end);
    return true;
}

template <int D, int NT, bool MX>
__global__ void __launch_bounds__(Geo<D, NT, MX>::THREADS, 1)
    decode_kernel(const __grid_constant__ DecodeArgs a, const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v)
{
    using G = Geo<D, NT, MX>;
    extern __shared__ uint8_t smem_dyn[];
    uint8_t *smem = smem_dyn + ((1024u - (smem_addr(smem_dyn) & 1023u)) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + G::BAR_OFF), *empty = full + MAX_STAGES;
    uint64_t *q_full = empty + MAX_STAGES, *q_empty = q_full + 2 * TEAMS;  // [TEAMS][2]
    int *bad = reinterpret_cast<int *>(smem + G::BAD_OFF);
    __shared__ long long scan[G::THREADS / 32];
    __shared__ Stretch first[TEAMS];
    __shared__ int abort_word;
    volatile int *abort_flag = &abort_word;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < G::STAGES; ++i) {
            mbar_init(&full[i], 2);
            mbar_init(&empty[i], TEAM);
        }
        for (int i = 0; i < 2 * TEAMS; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], TEAM);
        }
        abort_word = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async();
    }
    overlap_trigger();
    overlap_wait();

    // the list: every thread sums the tiles of some consecutive sequences
    const int per = (a.B + G::THREADS - 1) / G::THREADS;
    long long sum = 0;
    for (int b = tid * per; b < min(a.B, (tid + 1) * per); ++b)
        sum += places_of<G>(a, b);
    long long incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, o);
        incl += lane >= o ? v : 0;
    }
    if (lane == 31)
        scan[warp] = incl;
    __syncthreads();
    long long pre = incl - sum, total = 0;
    for (int w = 0; w < G::THREADS / 32; ++w) {
        pre += w < warp ? scan[w] : 0;
        total += scan[w];
    }
    total *= a.units;
    const long long share = share_of<G>(a, total);
    auto end_of = [&](int team) { return min(total, ((long long)team * gridDim.x + blockIdx.x + 1) * share); };
    if (tid < TEAMS)
        first[tid].t0 = first[tid].t1 = 0;
    __syncthreads();
#pragma unroll 1
    for (int k = 0; k < TEAMS; ++k) {
        const long long start = min(total, ((long long)k * gridDim.x + blockIdx.x) * share), end = end_of(k);
        if (start < end && pre * a.units <= start && start < (pre + sum) * a.units) {
            Stretch p;
            p.b = tid * per;
            long long base = pre;
            int n = places_of<G>(a, p.b);
            while (start >= (base + n) * a.units) {
                base += n;
                n = places_of<G>(a, ++p.b);
            }
            enter_sequence<G>(a, p, __ldcg(a.lens + p.b));
            p.u = (int)((start - base * a.units) / n);
            p.v = base * a.units + (long long)p.u * n;
            p.t0 = (int)max(0ll, start - p.v - G::START);
            cut<G>(a, p, end);
            if (a.whole && start > p.v && !advance<G>(a, p, end))
                p.t0 = p.t1 = 0;  // (the worker's places are the rest of another's unit)
            first[k] = p;
        }
    }
    // sequences without tiles: zeros, or NaN where the length cannot be
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        const int n = __ldcg(a.lens + b);
        if (n > 0 && n <= a.cap)
            continue;
        if (n != 0 && tid == 0)
            atomicCAS(a.err, 0, DEV_ERR_BOUNDS);
        const uint32_t v = n == 0 ? 0u : 0x7FC07FC0u;
        for (int i = tid; i < a.heads * D / 8; i += G::THREADS)
            reinterpret_cast<uint4 *>(a.out + b * a.out_ld)[i] = make_uint4(v, v, v, v);
    }
    __syncthreads();
    const int team = warp < G::WARPS ? warp / TEAM : (warp - G::WARPS) >> 1, worker = team * gridDim.x + blockIdx.x;
    const long long end = end_of(team);
    if (warp % TEAM == 0 && warp < G::WARPS && lane == 0)
        a.splits[worker] = {0, 0, 0, 0};  // (until the last stretch shows one)
    if (first[team].t1 <= first[team].t0)  // (none left, or no more than a unit's START places)
        return;
    Stretch at = first[team];
    const int page = 1 << a.page_log2, rows = min(page, G::TILE);  // rows of a TMA box

    if (warp >= G::WARPS) {
        // ------------------------------------------------------ tiles -> ring
        // A warp for each team's keys and one for its values: a copy costs its issuer about as long whatever its size,
        // and small pages take several.  A lane per page of a tile.  The table is read 32 pages at a time, a block
        // ahead: a tile's pages then cost a shuffle, where a load per tile would hold the loader up.
        const int pages = G::TILE / rows;
        const bool is_v = (warp - G::WARPS) & 1;
        const CUtensorMap *map = is_v ? &map_v : &map_k;
        const uint8_t *scales = is_v ? a.vs : a.ks;
        auto block = [&](int b, int k, int len) {  // the lane's entry of block k
            const int i = 32 * k + lane;
            return (long long)i << a.page_log2 < len ? __ldcg(a.table + (long long)b * a.max_pages + i) : 0;
        };
        int slot = team, n = 0;  // (every TEAMS-th slot is the team's); tiles so far
        uint32_t ph = 0;
        int held_b = -1, held_k = 0, held = 0, ahead = 0;
        int q_armed = -1;
        bool ok = true;
        for (int k = 0;; ++k) {  // stretches
            if (!is_v) {
                const int kvh = at.u / a.chunks, h0 = (at.u - kvh * a.chunks) * 8 * NT, heads = min(8 * NT, a.group - h0);
                uint64_t *bar = &q_full[2 * team + (k & 1)];
                if (!(ok = mbar_wait_sleep_warp(&q_empty[2 * team + (k & 1)], ((k >> 1) & 1) ^ 1, abort_flag, a.err, lane)))
                    break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar, heads * D * 2);
                    bulk_g2s(smem + G::Q_OFF + (2 * team + (k & 1)) * G::Q_B,
                             a.q + at.b * a.q_ld + ((long long)kvh * a.group + h0) * D, heads * D * 2, bar);
                    q_armed = k;
                }
                __syncwarp();
            }
            for (int t = at.t0; t < at.t1; ++t) {
                const int pg0 = (t * G::TILE) >> a.page_log2, bk = pg0 >> 5;
                if (at.b != held_b || bk != held_k) {
                    held = at.b == held_b && bk == held_k + 1 ? ahead : block(at.b, bk, at.len);
                    ahead = block(at.b, bk + 1, at.len);
                    held_b = at.b;
                    held_k = bk;
                }
                const int id = __shfl_sync(0xffffffffu, held, (pg0 & 31) + min(lane, pages - 1));
                const bool mine = lane < pages && (long long)(pg0 + lane) << a.page_log2 < at.len;
                const bool outside = id < 0 || id >= a.n_pages;
                if (!(ok = mbar_wait_sleep_warp(&empty[slot], ph ^ 1, abort_flag, a.err, lane)))
                    break;
                const uint32_t got = __ballot_sync(0xffffffffu, mine), wrong = __ballot_sync(0xffffffffu, mine && outside);
                if (lane == 0) {
                    if (wrong)
                        atomicCAS(a.err, 0, DEV_ERR_BOUNDS);
                    if (!is_v)
                        bad[slot] = wrong != 0;
                    mbar_arrive_expect_tx(&full[slot], __popc(got) * rows * (G::ROW_B + (MX ? D / 32 : 0)));
                }
                __syncwarp();
                if (mine) {
                    const int pg = outside ? 0 : id;  // (any page will do for one outside: the result is NaN)
                    const int kvh = at.u / a.chunks, off = (t * G::TILE) & (page - 1);
                    tma_4d(smem + (2 * slot + is_v) * G::TILE_B + lane * rows * G::ROW_B, map, 0, kvh * page + off, 0, pg,
                           &full[slot]);
                    if (MX) {
                        const long long row = (((long long)pg * a.kv + kvh) << a.page_log2) + off;
                        bulk_g2s(smem + G::SC_OFF + (2 * slot + is_v) * G::SC_B + lane * rows * (D / 32),
                                 scales + row * (D / 32), rows * (D / 32), &full[slot]);
                    }
                }
                ++n;
                if ((slot += TEAMS) >= G::STAGES) {
                    slot = team;
                    ph ^= 1;
                }
            }
            if (!ok || !advance<G>(a, at, end))
                break;
        }
        // every copy has landed before the CTA ends (bounded; slots whose other half never came run the limit out)
        if (lane == 0)
            for (int i = max(0, n - G::STAGES / TEAMS); i < n; ++i)
                if (!mbar_drain(&full[team + i % (G::STAGES / TEAMS) * TEAMS], i / (G::STAGES / TEAMS) & 1))
                    break;
        if (lane == 0)
            for (int k = max(0, q_armed - 1); k <= q_armed; ++k)
                mbar_drain(&q_full[2 * team + (k & 1)], (k >> 1) & 1);
        __syncwarp();
        return;
    }

    // ---------------------------------------------------------- products
    const int g = lane >> 2, qd = lane & 3, w4 = warp % TEAM;
    float *merge = reinterpret_cast<float *>(smem + G::MERGE_OFF) + team * 2 * NT * 8 * D;
    auto team_sync = [&] { asm volatile("barrier.cta.sync.aligned %0, %1;" ::"r"(1 + team), "n"(TEAM * 32) : "memory"); };
    const uint32_t ring = smem_addr(smem);
    constexpr float LOWERED = 1.f / (1 << (int)RAISED);
    int slot = team, part = 0;
    uint32_t ph = 0;
    Powers ref;
    bool alive = true, odd = false;
    State<D, NT> st;
    uint32_t qf[NT][D / 8];
    float mul[NT][2];
    for (int k = 0;; ++k) {  // stretches
        const int t0 = at.t0, t1 = at.t1;
        const int kvh = at.u / a.chunks, chunk = at.u - kvh * a.chunks;
        const int h0 = chunk * 8 * NT, heads = min(8 * NT, a.group - h0);
        const long long head = (long long)kvh * a.group + h0;
        alive = alive && __all_sync(0xffffffffu, mbar_wait(&q_full[2 * team + (k & 1)], (k >> 1) & 1, abort_flag, a.err)) != 0;
        const uint32_t q = ring + G::Q_OFF + (2 * team + (k & 1)) * G::Q_B;
        if (MX) {
            load_q_f16<D, NT>(a.scale, q, heads, g, qd, qf, mul);
        } else {
            load_q<D, NT>(q, heads, g, qd, qf);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                mul[nt][0] = mul[nt][1] = a.scale;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                st.m[nt][h] = -INFINITY;
                st.l[nt][h] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    st.o[i][nt][c] = 0.f;
        }
        ref = {0, false, true};
        __syncwarp();
        if (lane == 0 && alive)
            mbar_arrive(&q_empty[2 * team + (k & 1)]);
        bool wrong = !alive;
        for (int t = t0; t < t1; ++t) {
            // (after a wait that ran out the warp only keeps to the others' barriers; the rows become NaN)
            alive = alive && __all_sync(0xffffffffu, mbar_wait(&full[slot], ph, abort_flag, a.err)) != 0;
            wrong |= !alive || bad[slot] != 0;
            const uint32_t tile = ring + slot * 2 * G::TILE_B;
#pragma unroll 1
            for (int r = 16 * w4; r < G::TILE; r += 16 * TEAM) {
                const int n = min(16, at.len - t * G::TILE - r);
                if (!alive || n <= 0)
                    break;
                const int block = r / rows, r0 = r % rows;  // (a tile is blocks of `rows` rows, one or a part of a page)
                const uint32_t kb = tile + block * rows * G::ROW_B, vb = kb + G::TILE_B;
                if constexpr (MX) {
                    const uint32_t ksb = ring + G::SC_OFF + slot * 2 * G::SC_B + r * (D / 32);
                    tile_mx<D, NT>(st, qf, kb + r0 * G::ROW_B, vb + r0 * G::ROW_B, ksb, ksb + G::SC_B, n, mul, ref, lane);
                } else {
                    tile_bf16<D, NT>(st, qf, kb, vb, rows, r0, n, mul, g, qd);
                }
            }
            __syncwarp();
            if (lane == 0 && alive)
                mbar_arrive(&empty[slot]);
            if ((slot += TEAMS) >= G::STAGES) {
                slot = team;
                ph ^= 1;
            }
        }
        // The warps' parts: all come to the common maximum, the third's and the fourth's vectors go to the first and the
        // second, and the two sums meet in memory.
        // (maxima and sums lie in one of two places in turn: a warp may be one stretch ahead of the others' reads)
        float *ml = reinterpret_cast<float *>(smem + G::ML_OFF + (odd ? G::ML_B : 0)) + team * TEAM * NT * 8 * 2;
        odd = !odd;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float l = st.l[nt][h];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1)
                    l += __shfl_xor_sync(0xffffffffu, l, o);
                l *= MX ? LOWERED : 1.f;
                if (wrong)
                    l = __int_as_float(0x7FC00000);
                if (g == 0)
                    *reinterpret_cast<float2 *>(ml + ((w4 * NT + nt) * 8 + 2 * qd + h) * 2) = make_float2(st.m[nt][h], l);
            }
        team_sync();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float m = -INFINITY;
#pragma unroll
                for (int w = 0; w < TEAM; ++w)
                    m = fmaxf(m, ml[((w * NT + nt) * 8 + 2 * qd + h) * 2]);
                const float f = ex2(st.m[nt][h] - finite_base(m)) * (MX ? LOWERED : 1.f);
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    st.o[i][nt][h] *= f;
                    st.o[i][nt][2 + h] *= f;
                    if (MX) {
                        const float power = e8m0((ref.bytes >> (8 * (i / 2))) & 255);
                        st.o[i][nt][h] *= power;
                        st.o[i][nt][2 + h] *= power;
                    }
                }
            }
        float4 *mine = reinterpret_cast<float4 *>(merge + (w4 & 1) * NT * 8 * D) + lane;
        if (w4 >= 2) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mine[(i * NT + nt) * 32] = make_float4(st.o[i][nt][0], st.o[i][nt][1], st.o[i][nt][2], st.o[i][nt][3]);
        }
        team_sync();
        if (w4 < 2) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float4 x = mine[(i * NT + nt) * 32];
                    st.o[i][nt][0] += x.x, st.o[i][nt][1] += x.y, st.o[i][nt][2] += x.z, st.o[i][nt][3] += x.w;
                }
            __syncwarp();
            // in the order of heads and values: MMA i has a head's values 4 g + 2 (i & 1) and the next of 32 (MXFP8),
            // 8 g + 2 (i & 3) and the next of 64
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float *o = merge + (w4 * NT * 8 + nt * 8 + 2 * qd + h) * D;
#pragma unroll
                    for (int i = 0; i < D / 16; ++i)
                        *reinterpret_cast<float2 *>(o + (MX ? 32 * (i / 2) + 4 * g + 2 * (i & 1)
                                                            : 64 * (i / 4) + 8 * g + 2 * (i & 3))) =
                            make_float2(st.o[i][nt][h], st.o[i][nt][2 + h]);
                }
        }
        team_sync();
        const bool whole = t0 == 0 && t1 == at.nt;
        if (t0 == 0 && !whole && w4 == 0 && lane == 0)
            a.splits[worker] = {at.b, (int)head, heads * 2 + part, (int)((at.v + G::START + at.nt - 1) / share)};
        for (int i = w4 * 32 + lane; i < NT * D; i += TEAM * 32) {
            const int hd = i / (D / 8), d = i % (D / 8) * 8;
            if (hd >= heads)
                continue;
            float m = -INFINITY, l = 0.f, v[8] = {};
#pragma unroll
            for (int w = 0; w < TEAM; ++w)
                m = fmaxf(m, ml[(w * NT * 8 + hd) * 2]);
#pragma unroll
            for (int w = 0; w < TEAM; ++w) {
                const float2 x = *reinterpret_cast<const float2 *>(ml + (w * NT * 8 + hd) * 2);
                l = fmaf(x.y, ex2(x.x - finite_base(m)), l);
            }
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const float4 *o = reinterpret_cast<const float4 *>(merge + (w * NT * 8 + hd) * D + d);
                const float4 o0 = o[0], o1 = o[1];
                v[0] += o0.x, v[1] += o0.y, v[2] += o0.z, v[3] += o0.w;
                v[4] += o1.x, v[5] += o1.y, v[6] += o1.z, v[7] += o1.w;
            }
            if (whole) {
                const float inv = 1.f / l;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    v[k] *= inv;
                *reinterpret_cast<uint4 *>(a.out + at.b * a.out_ld + (head + hd) * D + d) = bf16x8(v);
            } else {
                const long long s = (2ll * worker + part) * 8 * NT + hd;
                float4 *o = reinterpret_cast<float4 *>(a.part_o + s * D + d);
                o[0] = make_float4(v[0], v[1], v[2], v[3]);
                o[1] = make_float4(v[4], v[5], v[6], v[7]);
                if (d == 0)
                    *reinterpret_cast<float2 *>(a.part_ml + 2 * s) = make_float2(m, l);
            }
        }
        part = 1;  // of a worker's stretches only the first and the last can be parts
        if (!advance<G>(a, at, end))
            break;
    }
}

// Joins the parts of a query head of the unit that starts with worker blockIdx.x and goes on with others; in the order of the
// parts, four warps taking them in turn.
template <int D, int NT>
__global__ void __launch_bounds__(128) join_kernel(const DecodeArgs a)
{
    constexpr int V = D / 32, WARPS = 4;  // values of a lane
    __shared__ float red[WARPS][D + 2];
    const int c0 = blockIdx.x, hd = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    overlap_trigger();
    overlap_wait();
    const int4 w = __ldcg(reinterpret_cast<const int4 *>(a.splits) + c0);
    const Split s{w.x, w.y, w.z, w.w};
    if (hd >= s.heads_part >> 1)
        return;
    float m = -INFINITY, l = 0.f, v[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        v[i] = 0.f;
#pragma unroll 4
    for (int c = c0 + warp; c <= s.last; c += WARPS) {
        const long long at = (2ll * c + (c == c0 ? s.heads_part & 1 : 0)) * 8 * NT + hd;
        const float2 x = __ldcg(reinterpret_cast<const float2 *>(a.part_ml + 2 * at));
        float o[V];
        if constexpr (V == 4) {
            const float4 u = __ldcg(reinterpret_cast<const float4 *>(a.part_o + at * D) + lane);
            o[0] = u.x, o[1] = u.y, o[2] = u.z, o[3] = u.w;
        } else {
            const float2 u = __ldcg(reinterpret_cast<const float2 *>(a.part_o + at * D) + lane);
            o[0] = u.x, o[1] = u.y;
        }
        const float next = fmaxf(m, x.x), base = finite_base(next), f = ex2(m - base), g = ex2(x.x - base);
        m = next;
        l = fmaf(l, f, x.y * g);
#pragma unroll
        for (int i = 0; i < V; ++i)
            v[i] = fmaf(v[i], f, o[i] * g);
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        red[warp][lane * V + i] = v[i];
    if (lane == 0) {
        red[warp][D] = m;
        red[warp][D + 1] = l;
    }
    __syncthreads();
    const int d = threadIdx.x;
    if (d >= D)
        return;
    m = -INFINITY;
#pragma unroll
    for (int i = 0; i < WARPS; ++i)
        m = fmaxf(m, red[i][D]);
    float sum = 0.f;
    l = 0.f;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) {
        const float f = ex2(red[i][D] - finite_base(m));
        l = fmaf(red[i][D + 1], f, l);
        sum = fmaf(red[i][d], f, sum);
    }
    a.out[s.b * a.out_ld + (long long)(s.head + hd) * D + d] = __bfloat16_as_ushort(__float2bfloat16_rn(sum / l));
}

// ---------------------------------------------------------------- host side

MoeStatus bad(MoeStatus s, const char *msg) { return (MoeStatus)set_last_error(s, msg); }

int head_tiles(int group) { return group <= 8 ? 1 : 2; }

// pages as {values of 128 bytes, rows of a page's heads, halves of a row, pages}
cudaError_t cache_map(CUtensorMap *m, const void *base, const MoeKvCache *c, int tile)
{
    auto enc = tensor_map_encoder();
    if (!enc)
        return cudaErrorNotSupported;
    const bool mx = c->type == MOE_ROWS_MXFP8;
    const int size = mx ? 1 : 2, inner = mx ? c->head_dim : 64, parts = c->head_dim / inner;
    const long long row = (long long)c->head_dim * size, rows = (long long)c->n_kv_heads * c->page_size;
    const cuuint64_t dims[4] = {(cuuint64_t)inner, (cuuint64_t)rows, (cuuint64_t)parts, (cuuint64_t)c->n_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)row, (cuuint64_t)(parts > 1 ? 128 : row), (cuuint64_t)(rows * row)};
    const cuuint32_t box[4] = {(cuuint32_t)inner, (cuuint32_t)(c->page_size < tile ? c->page_size : tile),
                               (cuuint32_t)parts, 1};
    const cuuint32_t step[4] = {1, 1, 1, 1};
    const CUresult r = enc(m, mx ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                           const_cast<void *>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           inner * size == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D, int NT, bool MX>
cudaError_t launch_decode(DecodeArgs &a, const MoeKvCache *cache, cudaStream_t st)
{
    using G = Geo<D, NT, MX>;
    CUtensorMap mk, mv;
    // Sequences are not shared between workers where the table holds at most 512 tokens (the lengths are known on the
    // device only), which saves the join: 2 us, and 3 us of the host's time for its launch.  Measured, shared and whole (us
    // in a graph; calls from Python): 56 heads on 8 of 128, one sequence of 256 tokens 8.0 and 6.2 (11.9 and 9.8), of 512
    // 7.7 and 8.6 (12.5 and 9.9), of 1000 7.9 and 13.2 (12.3 and 13.6); 88 of 1 to 256 20.5 and 19.0, of 1 to 500 26.0 and
    // 24.9; 32 of 1 to 500 16.0 and 15.9, of 1 to 1000 19.8 and 20.5.  One sequence of 512 so loses 0.9 us in a graph and
    // gains 2.6 where it is called.
    a.whole = a.cap <= 512;
    auto kern = decode_kernel<D, NT, MX>;
    static std::atomic<int> attr_set[MAX_DEVICES];
    cudaError_t e = smem_limit_once(attr_set, (const void *)kern, G::SMEM);
    if (e == cudaSuccess)
        e = cache_map(&mk, cache->k, cache, G::TILE);
    if (e == cudaSuccess)
        e = cache_map(&mv, cache->v, cache, G::TILE);
    if (e != cudaSuccess)
        return e;
    if ((e = launch_overlapped(kern, (unsigned)a.ctas, G::THREADS, G::SMEM, 1, st, a, mk, mv)) != cudaSuccess)
        return e;
    if (a.whole)  // nothing is shared
        return cudaSuccess;
    return launch_overlapped(join_kernel<D, NT>, dim3((unsigned)a.workers, 8 * NT), 128, 0, 1, st, a);
}

size_t part_bytes(int heads_of_part, int D)
{
    return (size_t)TEAMS * sm_count() * (2 * heads_of_part * (D + 2) * 4 + sizeof(Split));
}

bool heads_fit(int n_heads, int n_kv_heads)
{
    return n_heads >= 1 && n_heads <= ATTN_MAX_HEADS && n_kv_heads >= 1 && n_heads % n_kv_heads == 0;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" size_t moe_attention_decode_workspace_bytes(int B, int n_heads, int n_kv_heads, int head_dim)
{
    if (B < 1 || B > 65536 || !heads_fit(n_heads, n_kv_heads) || (head_dim != 64 && head_dim != 128))
        return 0;
    return part_bytes(8 * head_tiles(n_heads / n_kv_heads), head_dim);
}

extern "C" MoeStatus moe_attention_decode(const MoeKvCache *cache, const void *q, long long q_ld, int B, int n_heads,
                                          const int32_t *page_table, int max_pages, const int32_t *lens, float scale,
                                          void *out, long long out_ld, void *workspace, size_t ws_bytes,
                                          void *cuda_stream)
{
    char msg[160];
    const MoeStatus s = check_kv_cache(cache);
    if (s != MOE_OK)
        return s;
    const int D = cache->head_dim;
    if (B < 0 || B > 65536) {
        snprintf(msg, sizeof msg, "B = %d out of range [0, 65536]", B);
        return bad(MOE_EINVAL, msg);
    }
    if (!heads_fit(n_heads, cache->n_kv_heads)) {
        snprintf(msg, sizeof msg, "n_heads (%d) must be a multiple of the cache's %d heads and at most %d", n_heads,
                 cache->n_kv_heads, ATTN_MAX_HEADS);
        return bad(MOE_EINVAL, msg);
    }
    if (max_pages < 1 || (long long)max_pages * cache->page_size > 0x7FFFFFFFll)
        return bad(MOE_EINVAL, "moe_attention_decode: max_pages below 1, or 2^31 tokens and more");
    if (!(scale > 0.f) || !isfinite(scale * 1.4427f))
        return bad(MOE_EINVAL, "moe_attention_decode: scale must be finite and above 0");
    if (B == 0)
        return MOE_OK;
    if (!q || !page_table || !lens || !out)
        return bad(MOE_EINVAL, "moe_attention_decode: NULL q, page_table, lens or out");
    if (q_ld < (long long)n_heads * D || out_ld < (long long)n_heads * D)
        return bad(MOE_EINVAL, "moe_attention_decode: a row stride is below the row's values");
    if (!rows_16b(q, q_ld) || !rows_16b(out, out_ld) || (uintptr_t)page_table % 4 || (uintptr_t)lens % 4)
        return bad(MOE_EINVAL, "moe_attention_decode: rows must start on 16-byte boundaries, page_table and lens on "
                               "4-byte ones");
    const int group = n_heads / cache->n_kv_heads, nt = head_tiles(group);
    const size_t need = part_bytes(8 * nt, D);
    if (!workspace || ws_bytes < need || (uintptr_t)workspace % 256) {
        snprintf(msg, sizeof msg, "moe_attention_decode: workspace of %zu bytes, 256-byte aligned, is needed", need);
        return bad(MOE_EWORKSPACE, msg);
    }
    DecodeArgs a{};
    cudaError_t e = attention_error_flag(&a.err);
    if (e == cudaSuccess) {
        a.q = static_cast<const uint16_t *>(q);
        a.q_ld = q_ld;
        a.table = page_table;
        a.max_pages = max_pages;
        a.lens = lens;
        a.cap = (long long)max_pages * cache->page_size;
        a.B = B;
        a.heads = n_heads;
        a.kv = cache->n_kv_heads;
        a.group = group;
        a.chunks = (group + 8 * nt - 1) / (8 * nt);
        a.units = a.kv * a.chunks;
        a.n_pages = cache->n_pages;
        while ((1 << a.page_log2) < cache->page_size)
            ++a.page_log2;
        a.ks = static_cast<const uint8_t *>(cache->k_scales);
        a.vs = static_cast<const uint8_t *>(cache->v_scales);
        a.scale = scale * 1.44269504088896340736f;
        a.out = static_cast<uint16_t *>(out);
        a.out_ld = out_ld;
        a.ctas = gemm::sm_count();
        a.workers = TEAMS * a.ctas;
        a.part_o = static_cast<float *>(workspace);
        a.part_ml = a.part_o + (size_t)2 * a.workers * 8 * nt * D;
        a.splits = reinterpret_cast<Split *>(a.part_ml + (size_t)2 * a.workers * 8 * nt * 2);
        cudaStream_t st = (cudaStream_t)cuda_stream;
        const bool mx = cache->type == MOE_ROWS_MXFP8;
        if (D == 128)
            e = nt == 1 ? (mx ? launch_decode<128, 1, true>(a, cache, st) : launch_decode<128, 1, false>(a, cache, st))
                        : (mx ? launch_decode<128, 2, true>(a, cache, st) : launch_decode<128, 2, false>(a, cache, st));
        else
            e = nt == 1 ? (mx ? launch_decode<64, 1, true>(a, cache, st) : launch_decode<64, 1, false>(a, cache, st))
                        : (mx ? launch_decode<64, 2, true>(a, cache, st) : launch_decode<64, 2, false>(a, cache, st));
    }
    if (e != cudaSuccess) {
        snprintf(msg, sizeof msg, "decode attention launch: %s", cudaGetErrorString(e));
        return bad(MOE_ECUDA, msg);
    }
    return MOE_OK;
}
