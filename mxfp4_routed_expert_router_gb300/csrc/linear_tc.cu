// linear_tc.cu -- linear layers for more tokens than the weight stream of
// linear.cu is made for: y = x W^T on the 5th-generation tensor cores.
//
//   D[128 weight rows, up to 128 tokens] (FP32, tensor memory)
//       += A[128 rows, K] . B[tokens, K]^T
// A: weight rows.  4-bit weights are decoded by four warps (a lane per row) from
// the TILE-family store into tensor memory: MXFP4 to FP16 relative to the row's
// largest exponent, or to BF16 where a row's exponents span too widely; group-32
// INT4 to an exact FP16 pair hi + lo.  BF16 weights come by TMA into shared
// memory.  B: token rows by TMA, 128-byte-swizzled K-major tiles: the caller's
// BF16 rows with BF16 weights, else rows that a first kernel writes, with 4-bit
// weights in FP16 times a power of two per token.
//
// A CTA computes one tile (128 rows x up to 128 tokens x its K range) and two CTAs
// share an SM (half of its tensor memory each), so that the hand-offs, the first
// loads and the epilogue of one overlap the MMAs of the other.  A cluster of 1, 2,
// 4 or 8 CTAs splits K; its partial tiles meet in shared memory and each rank
// finishes a share of the tokens, in a fixed order.  Warps: 0 loads token tiles, 1
// issues the MMAs, 2 loads weight chunks, 4-11 decode (two groups of four, one per
// tensor-memory lane quadrant, taking the stages in turn) and then finish the tile.
// Weights and tokens come through rings of their own, as deep as the tile's size
// leaves room for: with few tokens the weight stream is what bounds a call, and
// its copies then run well ahead of the decoders.  The GEMM starts while the
// kernel that writes the token rows still runs and waits for it only before it
// reads them (overlap.cuh).  Every mbarrier wait is bounded (gemm_common.cuh).
//
// No unit is at its peak: with 512 and 2048 tokens of 7168 x 7168 the tensor pipe is
// active 0.4 to 0.66 of the time, L2 0.3 to 0.6 of its throughput, the path from L2 to
// the SMs 0.26 to 0.54, DRAM below 0.25.  BF16 weights, which have no decoder to wait
// for, are slower than MXFP4 ones: a 128 x 128 tile draws 16 KB of A and 16 KB of B
// per 64 of K from L2 (0.82 GB for 512 tokens, 3.3 GB for 2048; MXFP4 0.52 and 2.1 GB)
// through a ring of three such stages, so the latency of those loads is the likelier
// bound, with the tiles' balance (224 of them on 152 SMs) for 512 tokens.  With few
// tokens the roles' hand-offs bound it (a copy of the kernel without the decode and the
// MMAs still took 26 of 33 us), with INT4 weights the decoders (two operands to make).
// A tile is 128 tokens wide, as two CTAs share an SM's tensor memory (one CTA per SM with
// 256-wide tiles leaves nothing to run meanwhile); an MMA of 64 columns or fewer takes
// no longer than one of 64, so narrower tiles pay no less.
// Measured, us per call back to back with F32 rows, weights from HBM (linear.cu): MXFP4
// 7168 x 7168, 9 tokens 14.1, 32 14.8, 128 23.1, 512 49.8 (1.06 PFLOP/s), 2048 148
// (1.42), 36864 x 7168 with 2048 743 (1.46); group-32 INT4 7168 x 7168 21.8, 22.4, 31.1,
// 85, 284 (BF16 rows, which need no split of K, 244); BF16 19.0, 19.8, 26.1, 61, 166.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gemm_common.cuh"
#include "linear_internal.cuh"
#include "mx_decode.cuh"
#include "overlap.cuh"

namespace moe {

namespace {

using namespace gemm;

constexpr int N_WARPS = 12, THREADS = N_WARPS * 32;
constexpr int WARP_LOAD = 0, WARP_MMA = 1, WARP_WEIGHTS = 2, WARP_DEC = 4;  // (3 idles)
constexpr int DEC_GROUPS = 2;         // group g decodes the stages g, g + 2, ...
constexpr int NMAX = 128;             // tokens of a tile
constexpr int CHAIN_F32 = 512, CHAIN_F32_MX = 1152;  // MMAs into one accumulator for F32 rows (see launch_linear_gemm)
constexpr int A_MAX = 3;              // slots of the A ring (tensor memory): three with tiles of at most NHALF
constexpr int NHALF = 64;             // tokens, two with larger ones
constexpr int A_SLOT_COLS = 64;       // 128 16-bit values per lane
constexpr int TMEM_COLS = 256;        // half of the SM's: accumulator and A ring
static_assert(NMAX + 2 * A_SLOT_COLS <= TMEM_COLS && NHALF + A_MAX * A_SLOT_COLS <= TMEM_COLS, "tensor memory");
constexpr int A_TILE_BYTES = TILE_ROWS * HALF_K * 2;     // BF16 weights: 16 KB
// Shared memory: the token ring (a slot holds a stage's one or two swizzled tiles
// of tile_tokens x 128 bytes, with BF16 weights the A tile after it), then the ring
// of weight chunks.
constexpr int RING_BYTES = 108 * 1024;
constexpr int B_MAX = 12, W_MAX = 8;  // slots
constexpr int DONE = 12;              // barriers of finished stages
static_assert(DONE >= B_MAX, "see linear_tc_kernel");  // (B_MAX slots of one slice, half as many of two)
constexpr int BAR_OFF = RING_BYTES;
constexpr int N_BARS = B_MAX + 2 * W_MAX + A_MAX + DONE + 1;
constexpr int MISC_OFF = BAR_OFF + N_BARS * 8;
constexpr int TSC_OFF = MISC_OFF + 16;                   // exponents of the tile's tokens
constexpr int SMEM_BYTES = TSC_OFF + NMAX * 4 + 1024;    // + alignment slack
static_assert(2 * (SMEM_BYTES + 1024) <= 228 * 1024, "two CTAs per SM");
static_assert(NMAX * TILE_ROWS * 4 <= RING_BYTES, "a partial tile fits in the rings");

struct Args {
    const uint8_t *w;
    const uint8_t *row_base;  // FP16 operands: power of two (+ 127) of each row
    const float *xscale;      // FP16 operands: power of two of each token (2^-126 .. 2^114)
    int N, T, kchunks;
    int tile_tokens;          // tokens of a tile (a multiple of 16, at most NMAX), rows of a TMA box of B
    int ttiles;
    int b_slots, w_slots, w_off;  // ring slots, the weight ring's offset (bytes)
    void *y;
    long long y_ld;
    int y_f32, accumulate;
    int *err;
};

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void commit(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}

// K-major operand in shared memory, 128-byte swizzle, 8-row groups 1024 bytes apart
__device__ __forceinline__ uint64_t sw128(uint32_t saddr)
{
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

// kind::f16 with FP16 or BF16 A and B, FP32 D, both K-major, M = 128
__device__ __forceinline__ uint32_t instr_desc(bool bf16, int n)
{
    return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(TILE_ROWS >> 4) << 24);
}

// 64 values of K as four MMAs, A in tensor memory (8 columns per 16 values) or,
// with AS, in shared memory; the first adds to D only when acc0 != 0
template <bool AS>
__device__ __forceinline__ void mma64(uint32_t d, uint32_t a_tmem, uint64_t a_desc, uint64_t b, uint32_t idesc,
                                      uint32_t acc0)
{
    if (AS)
        asm volatile("{\n .reg .pred p, t;\n setp.ne.b32 p, %4, 0;\n setp.eq.b32 t, %4, %4;\n"
                     " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n"
                     " tcgen05.mma.cta_group::1.kind::f16 [%0], %5, %6, %3, t;\n"
                     " tcgen05.mma.cta_group::1.kind::f16 [%0], %7, %8, %3, t;\n"
                     " tcgen05.mma.cta_group::1.kind::f16 [%0], %9, %10, %3, t;\n}\n" ::"r"(d),
                     "l"(a_desc), "l"(b), "r"(idesc), "r"(acc0), "l"(a_desc + 2), "l"(b + 2), "l"(a_desc + 4),
                     "l"(b + 4), "l"(a_desc + 6), "l"(b + 6)
                     : "memory");
    else
        asm volatile("{\n .reg .pred p, t;\n setp.ne.b32 p, %4, 0;\n setp.eq.b32 t, %4, %4;\n"
                     " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
                     " tcgen05.mma.cta_group::1.kind::f16 [%0], [%5], %6, %3, t;\n"
                     " tcgen05.mma.cta_group::1.kind::f16 [%0], [%7], %8, %3, t;\n"
                     " tcgen05.mma.cta_group::1.kind::f16 [%0], [%9], %10, %3, t;\n}\n" ::"r"(d),
                     "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc0), "r"(a_tmem + 8), "l"(b + 2), "r"(a_tmem + 16),
                     "l"(b + 4), "r"(a_tmem + 24), "l"(b + 6)
                     : "memory");
}

// 16 tensor-memory columns of this warp's 32 lanes
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t v[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float v[16])
{
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i)
        v[i] = __uint_as_float(r[i]);
}

// {2^d, 2^d} in FP16, d in [-24, 0]
__device__ __forceinline__ uint32_t f16x2_pow2(int d)
{
    return (d >= -14 ? (uint32_t)(d + 15) << 10 : 1u << (d + 24)) * 0x10001u;
}

// 8 E2M1 codes -> 4 FP16 pairs times a power of two (exact)
__device__ __forceinline__ void decode_e2m1(uint32_t w, uint32_t s2, uint32_t out[4])
{
    uint32_t c[4];
    asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
        " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
        " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}"
        : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3])
        : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(out[i]) : "r"(c[i]), "r"(s2));
}

// One INT4 pair (codes in bits 0..3 and 16..19) as an exact FP16 pair hi + lo of
// s2 * (q - z): 0x6400 | q is 1024 + q, zz = {1024 + z, 1024 + z}
__device__ __forceinline__ void decode_i4(uint32_t w, uint32_t zz, uint32_t s2, uint32_t &hi, uint32_t &lo)
{
    uint32_t qz;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(qz) : "r"((w & 0x000F000Fu) | 0x64006400u), "r"(zz));
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(qz), "r"(s2));
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(lo) : "r"(qz), "r"(s2), "r"(hi ^ 0x80008000u));
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void store_y(const Args &a, long long at, float v)
{
    if (a.y_f32) {
        float *y = static_cast<float *>(a.y) + at;
        *y = a.accumulate ? *y + v : v;
    } else {
        static_cast<__nv_bfloat16 *>(a.y)[at] = __float2bfloat16_rn(v);
    }
}

// v * 2^e for a sum |v| < 2^47 of the MMAs and e = the row's exponent + the token's, -253 .. 241: neither power of two
// may be applied alone (v * 2^row or their product can leave FP32's range where the result does not), so e is
// split into one factor within the range and the rest of the same sign, which comes first.
__device__ __forceinline__ float scale_pow2(float v, int e)
{
    e = max(e, -252);  // (v * 2^e is 0 there already)
    const int c = min(max(e, -126), 127);
    return v * __int_as_float((127 + e - c) << 23) * __int_as_float((127 + c) << 23);
}

// This CTA's tile and its rank in the cluster.  Read afresh where they are needed
// again after the loops, so that no register holds them meanwhile.
struct Tile {
    int rt, tok0, nvalid, n_mma;
    uint32_t crank, csize;
};

__device__ __forceinline__ Tile tile_here(const Args &a)
{
    Tile t;
    uint32_t cta;
    asm volatile("mov.u32 %0, %%ctaid.x;" : "=r"(cta));
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(t.crank));
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(t.csize));
    const int item = cta / t.csize;
    t.rt = item / a.ttiles;
    t.tok0 = (item - t.rt * a.ttiles) * a.tile_tokens;
    t.nvalid = min(a.tile_tokens, a.T - t.tok0);
    t.n_mma = (t.nvalid + 15) & ~15;
    return t;
}

template <int OP, int WFMT>
__global__ void __launch_bounds__(THREADS, 2)
    linear_tc_kernel(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap map_b,
                     const __grid_constant__ CUtensorMap map_a)
{
    constexpr bool AS = WFMT == FMT_BF16;                            // A by TMA into shared memory
    constexpr int KST = (AS || OP == LIN_I4) ? HALF_K : CHUNK_K;     // K values per A stage
    constexpr int NSL = AS ? 1 : 2;                                  // 64-value token slices per slot of the token ring
    constexpr int BST = NSL * HALF_K / KST;                          // stages per slot (INT4: two)
    constexpr int NBLK = KST / 32;
    constexpr int CB = WFMT == FMT_INT4 ? CHUNK_I4_BYTES : CHUNK_MX_BYTES;
    extern __shared__ uint8_t smem_dyn[];
    uint8_t *smem = smem_dyn + ((1024u - (smem_addr(smem_dyn) & 1023u)) & 1023u);
    uint64_t *b_full = reinterpret_cast<uint64_t *>(smem + BAR_OFF), *w_full = b_full + B_MAX;
    uint64_t *w_empty = w_full + W_MAX, *a_full = w_empty + W_MAX, *done = a_full + A_MAX, *acc_full = done + DONE;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + MISC_OFF);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + MISC_OFF + 4);
    int *tsc = reinterpret_cast<int *>(smem + TSC_OFF);  // exponents of the tile's tokens

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Tile at0 = tile_here(a);
    const int rt = at0.rt, tok0 = at0.tok0, n_mma = at0.n_mma;
    const uint32_t crank = at0.crank, csize = at0.csize;
    const int c0 = (int)((long long)a.kchunks * crank / csize), c1 = (int)((long long)a.kchunks * (crank + 1) / csize);
    const int nst = (c1 - c0) * (CHUNK_K / KST);  // stages
    const uint32_t slice_bytes = (uint32_t)a.tile_tokens * HALF_K * 2;
    const uint32_t slot_bytes = NSL * slice_bytes + (AS ? A_TILE_BYTES : 0);

    if (tid == 0) {
        for (int i = 0; i < a.b_slots; ++i)
            mbar_init(&b_full[i], 1);
        for (int i = 0; i < a.w_slots; ++i) {
            mbar_init(&w_full[i], 1);
            mbar_init(&w_empty[i], KST == CHUNK_K ? 4 : 8);  // a chunk of two stages is read by both groups
        }
        for (int i = 0; i < A_MAX; ++i)
            mbar_init(&a_full[i], 4);
        for (int i = 0; i < DONE; ++i)
            mbar_init(&done[i], 1);
        mbar_init(acc_full, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async();
    }
    if (warp == WARP_MMA) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    // The MMAs of a stage are committed once, to the barrier of the stage: it frees
    // the stage's A slot and its part of the token slot.  Nobody waits for a stage
    // whose barrier could have come round again, which takes the end of stage + DONE:
    // the decoders' wait comes before they decode for stage + a_slots, and the
    // loader's before it loads for stage + BST * b_slots, which is stage + DONE or an
    // earlier one.  Nor does anybody skip a phase of a barrier that it waits for (it
    // could take the older one for it): decoder groups take every other chunk, and the
    // ring of chunks has an even number of slots.
    const uint32_t tmem = *tmem_slot;
    const int a_slots = a.tile_tokens <= NHALF ? A_MAX : 2;
    const uint32_t tmem_a = tmem + (a.tile_tokens <= NHALF ? NHALF : NMAX);

    if (warp == WARP_LOAD) {
        // ---------------------------------------------------------- token tiles -> ring
        overlap_wait();  // the token rows are written
        int it = 0, slot = 0, ds = BST - 1;
        uint32_t dph = 0;
        for (; it < nst / BST; ++it) {
            if (it >= a.b_slots) {  // the last stage that the slot held before
                if (!mbar_wait_sleep_warp(&done[ds], dph, abort_flag, a.err, lane))
                    break;
                if ((ds += BST) >= DONE) {
                    ds -= DONE;
                    dph ^= 1;
                }
            }
            if (lane == 0) {
                uint8_t *dst = smem + slot * slot_bytes;
                mbar_arrive_expect_tx(&b_full[slot], slot_bytes);
                if (AS) {  // the store seen as [row tiles * chunks * 2 halves * 128][64]
                    tma_2d(dst, &map_b, c0 * CHUNK_K + it * HALF_K, tok0, &b_full[slot]);
                    tma_2d(dst + slice_bytes, &map_a, 0, ((rt * a.kchunks + c0) * 2 + it) * TILE_ROWS, &b_full[slot]);
                } else {   // the rows seen as 64-value slices
                    tma_3d(dst, &map_b, 0, tok0, (c0 + it) * 2, &b_full[slot]);
                }
            }
            if (++slot == a.b_slots)
                slot = 0;
        }
        // every copy of an armed slot has landed before the CTA goes on (at once on
        // the normal path; bounded after an abort)
        if (lane == 0)
            for (int i = it > a.b_slots ? it - a.b_slots : 0; i < it; ++i)
                mbar_drain(&b_full[i % a.b_slots], (i / a.b_slots) & 1);
        __syncwarp();
    } else if (warp == WARP_WEIGHTS) {
        // ---------------------------------------------------------- weight chunks -> ring
        if (!AS) {
            const uint8_t *src = a.w + ((size_t)rt * a.kchunks + c0) * (size_t)CB;
            int c = 0, slot = 0;
            uint32_t ph = 0;
            for (; c < c1 - c0; ++c) {
                if (!mbar_wait_sleep_warp(&w_empty[slot], ph ^ 1, abort_flag, a.err, lane))
                    break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&w_full[slot], CB);
                    bulk_g2s(smem + a.w_off + slot * CB, src + (size_t)c * CB, CB, &w_full[slot]);
                }
                if (++slot == a.w_slots) {
                    slot = 0;
                    ph ^= 1;
                }
            }
            if (lane == 0)
                for (int i = c > a.w_slots ? c - a.w_slots : 0; i < c; ++i)
                    mbar_drain(&w_full[i % a.w_slots], (i / a.w_slots) & 1);
        }
        __syncwarp();
    } else if (warp == WARP_MMA) {
        // ---------------------------------------------------------- MMAs
        // The whole warp runs the loop and one elected lane issues: the operands are
        // then computed in converged code (measured: 26 cycles an MMA against 49 from
        // a loop that one lane runs).
        uint32_t elected;
        asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(elected));
        auto wait = [&](uint64_t *bar, uint32_t par) {
            return __all_sync(0xffffffffu, mbar_wait(bar, par, abort_flag, a.err)) != 0;
        };
        const uint64_t desc0 = sw128(smem_addr(smem)), slice = (uint64_t)(slice_bytes >> 4);
        const uint32_t idesc = instr_desc(OP == LIN_BF16, n_mma);
        uint64_t bd = desc0;
        uint32_t at = tmem_a, aph = 0, bph = 0;
        int as = 0, ds = 0, slot = 0;
        for (int st = 0; st < nst; ++st) {
            if (!AS && !wait(&a_full[as], aph))
                break;
            const int half = BST == 2 ? st & 1 : 0;
            if (half == 0 && !wait(&b_full[slot], bph))
                break;
            fence_after();
            if (elected) {
                if (AS) {
                    mma64<true>(tmem, 0, bd + slice, bd, idesc, st);
                } else if (OP == LIN_I4) {
                    mma64<false>(tmem, at, 0, bd + half * slice, idesc, st);
                    mma64<false>(tmem, at + 32, 0, bd + half * slice, idesc, 1u);
                } else {
                    mma64<false>(tmem, at, 0, bd, idesc, st);
                    mma64<false>(tmem, at + 32, 0, bd + slice, idesc, 1u);
                }
                commit(&done[ds]);
            }
            __syncwarp();
            if (++ds == DONE)
                ds = 0;
            if (half == BST - 1) {
                bd += (uint64_t)(slot_bytes >> 4);
                if (++slot == a.b_slots) {
                    slot = 0;
                    bph ^= 1;
                    bd = desc0;
                }
            }
            at += A_SLOT_COLS;
            if (++as == a_slots) {
                as = 0;
                aph ^= 1;
                at = tmem_a;
            }
        }
        // also after an abort: what was issued has completed before the tensor memory
        // is freed and the rings reused
        if (elected) {
            commit(acc_full);
            mbar_drain(acc_full, 0);
        }
        __syncwarp();
    } else if (warp >= WARP_DEC) {
        // ---------------------------------------------------------- decode
        const int q = warp & 3, grp = (warp - WARP_DEC) >> 2, r = 32 * q + lane;  // lane quadrant; row of the tile
        const uint32_t tlane = (uint32_t)(32 * q) << 16;
        bool ok = true;
        if (!AS) {
            const int rb = OP == LIN_BF16 ? 127 : (int)__ldg(a.row_base + rt * TILE_ROWS + r);
            constexpr int STEP = KST == CHUNK_K ? DEC_GROUPS : 1;  // chunks from one stage of the group to its next
            int slot = KST == CHUNK_K ? grp : 0;
            uint32_t ph = 0;
            const bool second = KST < CHUNK_K && grp == 1;         // this group decodes the chunks' second halves
            int as = grp;                                          // the stage's A slot
            int ds = (grp + a_slots) & 1;                          // barrier of the stage that the slot held before
            uint32_t dph = 0;
            for (int st = grp; st < nst; st += DEC_GROUPS) {
                if (!(ok = mbar_wait_warp(&w_full[slot], ph, abort_flag, a.err, lane)))
                    break;
                const uint8_t *ch = smem + a.w_off + slot * CB;
                uint4 code[NBLK];
                uint32_t sc[NBLK];
#pragma unroll
                for (int b = 0; b < NBLK; ++b) {
                    const int blk = (second ? 2 : 0) + b;
                    if (OP == LIN_I4) {
                        code[b] = *reinterpret_cast<const uint4 *>(ch + (blk * TILE_ROWS + r) * 16);
                        sc[b] = (uint32_t)*(reinterpret_cast<const uint16_t *>(ch + CHUNK_MX_CODE_BYTES) +
                                            blk * TILE_ROWS + r) |
                                (uint32_t)ch[CHUNK_MX_CODE_BYTES + CHUNK_I4_SCALE_BYTES + blk * TILE_ROWS + r] << 16;
                    } else if (OP == LIN_F16) {
                        code[b] = *reinterpret_cast<const uint4 *>(ch + (blk * TILE_ROWS + r) * 16);
                        sc[b] = ch[CHUNK_MX_CODE_BYTES + blk * TILE_ROWS + r];
                    } else {
                        code[b] = *reinterpret_cast<const uint4 *>(ch + (blk >> 1) * (CHUNK_MX_CODE_BYTES / 2) +
                                                                   r * 32 + (blk & 1) * 16);
                        sc[b] = ch[CHUNK_MX_CODE_BYTES + r * 4 + blk];
                    }
                }
                __syncwarp();  // the stage's codes are in registers
                if (lane == 0)
                    mbar_arrive(&w_empty[slot]);
                if ((slot += STEP) >= a.w_slots) {
                    slot -= a.w_slots;
                    ph ^= 1;
                }
                // The first block of the stage is decoded before the wait for its A slot, so that
                // less lies between the end of the MMAs that used it and those that wait for it
                // (INT4 7168 x 18432, 512 tokens, K whole: 221 -> 199 us; more blocks gain nothing more).
                uint32_t o[16], lo[16];
                auto decode = [&](int b, uint32_t *hi, uint32_t *rest) {
                    const uint32_t w[4] = {code[b].x, code[b].y, code[b].z, code[b].w};
                    if (OP == LIN_I4) {
                        // relative to the row's base (the scale then lies below 2^12, and is exact:
                        // launch_row_base keeps weights where one is not away from this kernel)
                        const float sf = __half2float(__ushort_as_half((unsigned short)(sc[b] & 0xFFFFu))) *
                                         __int_as_float((254 - rb) << 23);
                        const uint32_t s2 = (uint32_t)__half_as_ushort(__float2half_rn(sf)) * 0x10001u;
                        const uint32_t zz = (0x6400u + (sc[b] >> 16)) * 0x10001u;
#pragma unroll
                        for (int c = 0; c < 4; ++c)
#pragma unroll
                            for (int p = 0; p < 4; ++p)
                                decode_i4(w[c] >> (4 * p), zz, s2, hi[4 * c + p], rest[4 * c + p]);
                    } else if (OP == LIN_F16) {
                        int d = (int)sc[b] - rb;
                        d = d < -24 ? -24 : (d > 0 ? 0 : d);  // (blocks past K, whose codes are 0)
                        const uint32_t s2 = f16x2_pow2(d);
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            decode_e2m1(w[c], s2, hi + 4 * c);
                    } else {
                        const uint32_t s2 = e8m0_to_bf16x2(sc[b]);
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            decode_word(w[c], s2, hi + 4 * c);
                    }
                };
                decode(0, o, lo);
                if (st >= a_slots) {
                    if (!(ok = mbar_wait_warp(&done[ds], dph, abort_flag, a.err, lane)))
                        break;
                    if ((ds += DEC_GROUPS) >= DONE) {
                        ds -= DONE;
                        dph ^= 1;
                    }
                }
                fence_after();
                const uint32_t dst = tmem_a + tlane + as * A_SLOT_COLS;
#pragma unroll
                for (int b = 0; b < NBLK; ++b) {
                    if (b > 0)
                        decode(b, o, lo);
                    if (OP == LIN_I4)
                        tmem_st16(dst + 32 + b * 16, lo);
                    tmem_st16(dst + b * 16, o);
                }
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&a_full[as]);
                if ((as += DEC_GROUPS) >= a_slots)
                    as -= a_slots;
            }
        }
        // ---------------------------------------------------------- the tile's sums
        overlap_trigger();
        overlap_wait();
        const Tile at1 = tile_here(a);
        const int rt = at1.rt, tok0 = at1.tok0, nvalid = at1.nvalid, n_mma = at1.n_mma;
        const uint32_t csize = at1.csize;
        if (OP != LIN_BF16) {  // (every warp writes the same values and reads its own)
            for (int i = lane; i < nvalid; i += 32)
                tsc[i] = (__float_as_int(__ldcg(a.xscale + tok0 + i)) >> 23) - 127;
            __syncwarp();
        }
        if (ok && mbar_wait_sleep_warp(acc_full, 0, abort_flag, a.err, lane)) {
            fence_after();
            const int n = rt * TILE_ROWS + r;
            const int we = OP == LIN_BF16 ? 0 : (int)__ldg(a.row_base + rt * TILE_ROWS + r) - 127;
            float *part = reinterpret_cast<float *>(smem) + r;  // [token][128]: the rings are free
            for (int c = 16 * grp; c < n_mma; c += 16 * DEC_GROUPS) {
                float v[16];
                tmem_ld16(tmem + tlane + c, v);
                if (csize > 1) {
#pragma unroll
                    for (int j = 0; j < 16; ++j)  // (columns past nvalid: inside the tile's room, not read)
                        part[(c + j) * TILE_ROWS] = v[j];
                } else if (n < a.N) {
                    const long long at = (long long)(tok0 + c) * a.y_ld + n;
                    if (OP != LIN_BF16)
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            v[j] = scale_pow2(v[j], we + tsc[c + j]);
                    if (a.accumulate) {  // all loads before the first store
                        float old[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            old[j] = c + j < nvalid ? static_cast<const float *>(a.y)[at + j * a.y_ld] : 0.f;
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            v[j] += old[j];
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (c + j < nvalid) {
                            if (a.y_f32)
                                static_cast<float *>(a.y)[at + j * a.y_ld] = v[j];
                            else
                                static_cast<__nv_bfloat16 *>(a.y)[at + j * a.y_ld] = __float2bfloat16_rn(v[j]);
                        }
                }
            }
        }
        fence_before();
    }

    __syncwarp();
    const Tile at2 = tile_here(a);
    if (at2.csize > 1) {
        const int rt = at2.rt, tok0 = at2.tok0, nvalid = at2.nvalid;
        const uint32_t crank = at2.crank, csize = at2.csize;
        cluster_sync();
        // rank r finishes tokens r, r + csize, ... of the tile: a warp per token, four rows a lane
        if (!*abort_flag) {
            const uint32_t part = smem_addr(smem);
            for (int t = crank + csize * warp; t < nvalid; t += csize * N_WARPS) {
                const uint32_t local = part + (t * TILE_ROWS + lane * 4) * 4;
                float4 f[8];
#pragma unroll
                for (uint32_t rk = 0; rk < 8; ++rk)  // all ranks' loads in flight
                    if (rk < csize) {
                        uint32_t remote;
                        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rk));
                        asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                                     : "=f"(f[rk].x), "=f"(f[rk].y), "=f"(f[rk].z), "=f"(f[rk].w)
                                     : "r"(remote));
                    }
                float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (uint32_t rk = 0; rk < 8; ++rk)
                    if (rk < csize)
                        o[0] += f[rk].x, o[1] += f[rk].y, o[2] += f[rk].z, o[3] += f[rk].w;
                // row exponents (+ 127) of the lane's four rows
                const uint32_t rb4 = OP == LIN_BF16 ? 0u : __ldg(reinterpret_cast<const uint32_t *>(a.row_base) +
                                                                 rt * (TILE_ROWS / 4) + lane);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int n = rt * TILE_ROWS + lane * 4 + j;
                    if (OP != LIN_BF16)
                        o[j] = scale_pow2(o[j], (int)(rb4 >> (8 * j) & 255u) - 127 + tsc[t]);
                    if (n < a.N)
                        store_y(a, (long long)(tok0 + t) * a.y_ld + n, o[j]);
                }
            }
        }
        __syncwarp();
        cluster_sync();  // partial sums stay in place until every rank has read them
    }
    __syncthreads();
    if (warp == WARP_MMA) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
    }
}

// Token rows of the GEMM, one CTA per token: FP16 x * 2^-e (a power of two per
// token: the largest |x| lands in [2^14, 2^15); exact within 2^-29 of it) with
// scale[t] = 2^e, or BF16 (of MXFP8 rows).
__global__ void __launch_bounds__(1024) linear_rows_kernel(const void *x, const uint8_t *xscales, long long x_ld,
                                                          int x_mx, int K, int kpad, int bf16, uint16_t *out,
                                                          float *scale)
{
    __shared__ uint32_t red[32];
    const long long t = blockIdx.x;
    const int nt = blockDim.x;
    overlap_trigger();  // the GEMM starts on the weights
    overlap_wait();
    auto load = [&](int v, float f[8]) {
        if (x_mx) {
            const uint2 u = __ldcg(reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(x) + t * x_ld) + v);
            const int e = __ldcg(xscales + t * (K / 32) + v / 4);
            const float s = e == 255 ? __int_as_float(0x7FC00000) : __int_as_float(e ? e << 23 : 0x400000);
            const uint32_t w[2] = {u.x, u.y};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint16_t c = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
                uint32_t h;
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
                const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&h));
                f[2 * i] = p.x * s;
                f[2 * i + 1] = p.y * s;
            }
        } else {
            const uint4 u = __ldcg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(x) + t * x_ld) + v);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
        }
    };
    const int nv = K / 8;
    float mul = 1.f;
    if (!bf16) {
        float m = 0.f;  // (NaN is left out and stays NaN in FP16)
        for (int v = threadIdx.x; v < nv; v += nt) {
            float f[8];
            load(v, f);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                m = fmaxf(m, fabsf(f[i]));
        }
        uint32_t b = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
        if ((threadIdx.x & 31) == 0)
            red[threadIdx.x >> 5] = b;
        __syncthreads();
        b = 0;
        for (int i = 0; i < nt / 32; ++i)
            b = max(b, red[i]);
        const int e = max((int)(b >> 23) - 141, -126);
        mul = __int_as_float((127 - e) << 23);
        if (threadIdx.x == 0)
            scale[t] = __int_as_float((127 + e) << 23);
    }
    for (int v = threadIdx.x; v < kpad / 8; v += nt) {
        float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};  // (zeros up to a whole chunk)
        uint32_t o[4];
        if (v < nv)
            load(v, f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (bf16) {
                const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                o[i] = *reinterpret_cast<const uint32_t *>(&p);
            } else {
                const __half2 p = __floats2half2_rn(f[2 * i] * mul, f[2 * i + 1] * mul);
                o[i] = *reinterpret_cast<const uint32_t *>(&p);
            }
        }
        reinterpret_cast<uint4 *>(out + t * (long long)kpad)[v] = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// ------------------------------------------------------------------ host side

// [rows][cols] 16-bit values with a row pitch in bytes, boxes of 64 x box_rows
cudaError_t rows_map(CUtensorMap *m, const void *base, long long rows, int cols, long long pitch, int box_rows)
{
    auto enc = tensor_map_encoder();
    if (!enc)
        return cudaErrorNotSupported;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)pitch};
    cuuint32_t box[2] = {HALF_K, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int OP, int WFMT>
cudaError_t launch_cfg(const Args &a, const CUtensorMap &mb, const CUtensorMap &ma, int grid, int cluster,
                       cudaStream_t st)
{
    auto kern = linear_tc_kernel<OP, WFMT>;
    static std::atomic<int> attr_set[MAX_DEVICES];
    const cudaError_t e = smem_limit_once(attr_set, (const void *)kern, SMEM_BYTES);
    if (e != cudaSuccess)
        return e;
    return launch_overlapped(kern, (unsigned)grid, THREADS, SMEM_BYTES, cluster, st, a, mb, ma);
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace

size_t linear_gemm_workspace(int K, int T)
{
    const size_t kpad = (size_t)((K + CHUNK_K - 1) & ~(CHUNK_K - 1));
    return align256((size_t)T * kpad * 2) + align256((size_t)T * 4);
}

cudaError_t launch_linear_gemm(const LinearGemm &g, cudaStream_t st)
{
    Args a{};
    a.w = g.w->base;
    a.row_base = g.w->row_base;
    a.N = g.N;
    a.T = g.T;
    a.kchunks = g.w->kchunks;
    a.ttiles = (g.T + NMAX - 1) / NMAX;
    a.tile_tokens = ((g.T + a.ttiles - 1) / a.ttiles + 15) & ~15;
    a.ttiles = (g.T + a.tile_tokens - 1) / a.tile_tokens;
    a.y = g.y;
    a.y_ld = g.y_ld;
    a.y_f32 = g.y_f32;
    a.accumulate = g.accumulate;
    a.err = g.err;
    const bool bf16 = g.op == LIN_BF16;
    // the rings: enough token slots to cover their loads, the rest for weight chunks
    const int nsl = g.fmt == FMT_BF16 ? 1 : 2;
    const int slot_bytes = nsl * a.tile_tokens * HALF_K * 2 + (g.fmt == FMT_BF16 ? A_TILE_BYTES : 0);
    if (g.fmt == FMT_BF16) {
        a.b_slots = RING_BYTES / slot_bytes < B_MAX ? RING_BYTES / slot_bytes : B_MAX;
        a.w_slots = 0;
    } else {
        a.b_slots = (a.tile_tokens <= 32 ? B_MAX : a.tile_tokens <= 64 ? 8 : a.tile_tokens <= 96 ? 6 : 4) / nsl;
        a.w_off = a.b_slots * slot_bytes;
        a.w_slots = (RING_BYTES - a.w_off) / g.w->chunk_bytes;
        if (a.w_slots > W_MAX)
            a.w_slots = W_MAX;
        if (g.op != LIN_I4)
            a.w_slots &= ~1;  // (see linear_tc_kernel; with INT4 both groups read every chunk)
    }
    CUtensorMap mb, ma;
    cudaError_t e;
    const bool rows_written = g.fmt != FMT_BF16 || g.x_mx;
    const int kpad = (g.K + CHUNK_K - 1) & ~(CHUNK_K - 1);
    if (!rows_written) {
        e = rows_map(&mb, g.x, g.T, g.K, g.x_ld * 2, a.tile_tokens);
    } else {
        uint16_t *rows = reinterpret_cast<uint16_t *>(g.workspace);
        float *scale = reinterpret_cast<float *>(g.workspace + align256((size_t)g.T * kpad * 2));
        if ((e = launch_overlapped(linear_rows_kernel, g.T, g.T <= 2 * sm_count() ? 1024 : 256, 0, 1, st, g.x, g.xscales,
                                   g.x_ld, (int)g.x_mx, g.K, kpad, (int)bf16, rows, scale)) != cudaSuccess)
            return e;
        a.xscale = scale;
        e = g.fmt == FMT_BF16 ? rows_map(&mb, rows, g.T, kpad, (long long)kpad * 2, a.tile_tokens)
                              : make_map_3d(&mb, rows, g.T, kpad, a.tile_tokens, nsl);
    }
    if (e != cudaSuccess)
        return e;
    ma = mb;
    if (g.fmt == FMT_BF16 &&
        (e = rows_map(&ma, g.w->base, (long long)g.w->row_tiles * g.w->kchunks * 2 * TILE_ROWS, HALF_K, HALF_K * 2,
                      TILE_ROWS)) != cudaSuccess)
        return e;
    // K split over a cluster while two CTAs per SM are not all in use
    const long long items = (long long)g.w->row_tiles * a.ttiles;
    if (items > (1 << 28))
        return cudaErrorInvalidValue;
    int cluster = 1;
    while (cluster < 8 && items * cluster * 2 <= 2ll * sm_count() && cluster * 2 <= a.kchunks)
        cluster *= 2;
    // An MMA adds to its FP32 accumulator by truncation, half of a last place on average and always towards zero, so
    // that a long chain drifts: error against 64 bits at K = 18432 in one chain 2.1e-5 of the norm (BF16), 4.0e-5
    // (INT4, two MMAs per 16 values) where an FP32 sum is 2e-6 off.  BF16 rows round by 100 times that; for F32 rows K
    // is split further, as far as a cluster goes, and the parts add up rounded to nearest: 5e-6 (INT4 512 x 7168 x
    // 18432 199 -> 224 us, BF16 142 -> 174).  MXFP4's products have 10 bits and lose less: 3.4e-6 with scales within
    // 2^4 of each other, 1.5e-5 at most, at K = 18432, which is left whole (114 us; 164 in four parts).
    const int chain = g.w->kchunks * (CHUNK_K / 16) * (g.op == LIN_I4 ? 2 : 1);
    const int chain_most = g.op == LIN_F16 ? CHAIN_F32_MX : CHAIN_F32;
    while (g.y_f32 && cluster < 8 && chain > chain_most * cluster && cluster * 2 <= a.kchunks)
        cluster *= 2;
    const int grid = (int)items * cluster;
    switch (g.op) {
    case LIN_F16: return launch_cfg<LIN_F16, FMT_MXFP4>(a, mb, ma, grid, cluster, st);
    case LIN_I4: return launch_cfg<LIN_I4, FMT_INT4>(a, mb, ma, grid, cluster, st);
    default:
        return g.fmt == FMT_BF16 ? launch_cfg<LIN_BF16, FMT_BF16>(a, mb, ma, grid, cluster, st)
                                 : launch_cfg<LIN_BF16, FMT_MXFP4>(a, mb, ma, grid, cluster, st);
    }
}

}  // namespace moe
