// attention_prompt.cu -- causal attention within packed prompts (moe_attention_prompt, include/moe.h) on the
// 5th-generation tensor cores.
//
//   S = Q K^T,  P = 2^(scale log2(e) S - m),  O = sum of P V over the key tiles,  out = O / sum of P
// with m a row's running maximum: one pass over the keys, nothing of S or P leaves the SM.
//
// A CTA has 256 rows as two tiles of 128: 128 / group tokens (rounded down) of a tile times the `group` query heads of
// one key head, so that short sequences fill tiles too and a key tile is loaded once for all heads that read it.  It
// goes over the keys of its sequence in tiles of 128 up to its last token.  Warps: 0-3 and 4-7 the softmax of either
// tile (a thread per row), 8 issues the MMAs, 9 loads by TMA, 10 and 11 look after values that no row may see (below).
// Tensor memory: S of both tiles (128 columns each; P overwrites its tile's S as BF16, but for heads of 64) and O of
// both.  MMAs go in the order S0 S1 | PV0 S0' | PV1 S1' | ..., so that one tile's softmax runs under the other tile's
// products, and a tile's next S, which comes after its PV in the same queue, says that this PV is done: O may then be
// touched without a wait.  Heads of 64, whose products take half as long as the softmax, leave room for P of its own:
// S0' PV0 | S1' PV1, with S' under the softmax of S.
// The maximum in use is kept until a row exceeds it by 2^8 (P is then up to 2^8, in BF16's and FP32's range alike):
// rescaling O in tensor memory, which would be needed in every tile, becomes rare.
//
// Measured (device time): 8192 rows, 64 heads on 8 of 128, 670 to 706 us (1.1 TFLOP: 1,640 to 1,560 TFLOP/s, 0.84 to
// 0.80 of a cuBLAS burst, by how far the card's power limit has brought the clock down; 4 key heads with pauses 1,700).
// A key tile takes 2,900 cycles for 2,048 of MMAs: a tile's softmax (load 150, maximum 400, exponentials 900, store
// 110) and its own products (1,024 and 250 of latency) follow each other, and two tiles fill a third of each other's
// gaps.  Tried without gain: P announced by halves; the exponentials with the old maximum while the new one is found;
// two threads to a row (16 warps, a barrier of two per tile: 704 us for 673); rows that leave by TMA or, over shared
// memory, by whole lines.  A new item costs 2 to 3 us beside its key tiles, so that short prompts get less (15 prompts
// of 1 to 3001 rows, 56 heads on 8: 500 to 510 us for 650 GFLOP).  Heads of 64: 8192 rows, 32 heads on 4, 250 us, bound by
// the latency of the softmax (two warps a scheduler; issue slots 51 %, exponentials 49 % of their pipe, tensor 46 %).
//
// Masked values: P is 0 there, but 0 * inf is not.  Two warps clear the rows of V past the sequence's end, and values
// that are not finite in tiles that some row must not see in full; rows that may see such a value get it added at the
// end.  A CTA per SM goes over its items (two tiles of a key head) one after the other, without a gap: the next item's
// tiles are on their way and its first S is computed while the last one's rows are written.
#include <math.h>
#include <stdio.h>

#include "attention_internal.cuh"
#include "gemm_common.cuh"
#include "mx_encode.cuh"
#include "overlap.cuh"

namespace moe {

namespace {

using namespace gemm;

constexpr int BM = 128, BN = 128;    // rows of a tile, keys of a tile
constexpr int THREADS = 384;
constexpr int WARP_MMA = 8, WARP_LOAD = 9, WARP_GUARD = 10;
constexpr int GUARDS = 2;
constexpr int TMEM_COLS = 512;
// Registers: 168 a thread at launch; the warps that do not compute rows give some of theirs to those that do.
constexpr int SOFTMAX_REGS = 208, OTHER_REGS = 80;
static_assert(256 * SOFTMAX_REGS + 128 * OTHER_REGS <= 168 * THREADS, "the launch's registers");
constexpr float GROWTH = 8.f;        // log2 by which a row's maximum may exceed the one in use

struct PromptArgs {
    const int32_t *offsets;
    int n_seqs, T, max_items;
    int heads, kv, group, tile_tokens;  // tokens of a tile
    const uint16_t *v;
    long long v_ld;
    float scale;                        // times log2(e)
    uint16_t *out;
    long long out_ld;
    bool wide_out;                      // rows of out start on 32-byte boundaries
    int *err;
};

template <int D> struct PGeo {
    static constexpr int TILE_B = 128 * D * 2;              // 128 rows
    // Tensor memory: S, P and O of the two tiles.  With heads of 64 there is room for P beside S, so that a tile's next
    // S need not wait for the product that reads its P.
    static constexpr bool APART = D == 64;
    static constexpr int P_COL = APART ? 2 * BN : 0, P_STEP = APART ? BN / 2 : BN;
    static constexpr int O_COL = APART ? 3 * BN : 2 * BN;
    static_assert(O_COL + 2 * D <= TMEM_COLS, "tensor memory");
    static constexpr int SLOTS = D == 128 ? 5 : 8;          // key and value tiles
    static constexpr int RING_OFF = 2 * TILE_B;
    static constexpr int BAR_OFF = RING_OFF + SLOTS * TILE_B;
    static constexpr int N_BARS = 4 * SLOTS + 8 + 2 + 4 + 1;
    static constexpr int SMEM = BAR_OFF + N_BARS * 8 + 1024;  // + alignment slack
    static_assert(SMEM <= 226 * 1024, "shared memory");
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two floats in one register pair: one instruction for both
__device__ __forceinline__ uint64_t pack2(float x, float y)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}

__device__ __forceinline__ float2 unpack2(uint64_t v)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// The largest of a row's 128 scores
__device__ __forceinline__ float row_max(const uint32_t (&s)[BN])
{
    float m[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m[i] = fmaxf(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1]));
#pragma unroll
    for (int c = 16; c < BN; c += 16)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            m[i] = max3(m[i], __uint_as_float(s[c + 2 * i]), __uint_as_float(s[c + 2 * i + 1]));
    m[0] = max3(m[0], m[1], m[2]);
    m[3] = max3(m[3], m[4], m[5]);
    return max3(max3(m[0], m[3], m[6]), m[7], m[7]);
}

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void commit(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}

// K-major operand, 128-byte swizzle, 8-row groups 1024 bytes apart
__device__ __forceinline__ uint64_t desc_k(uint32_t saddr)
{
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

// The other major: 64 values of N side by side in 128 bytes, rows of K 128 bytes apart (8-row groups 1024), the next 64
// values of N a tile half (16 KB) on
__device__ __forceinline__ uint64_t desc_n(uint32_t saddr)
{
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (1024ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

// kind::f16, BF16 operands, FP32 accumulator, M = 128
constexpr uint32_t instr_desc(int n, bool b_n_major)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | (b_n_major ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(BM >> 4) << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                 " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(acc)
                 : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                 " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
                 "r"(a), "l"(b), "r"(idesc), "r"(acc)
                 : "memory");
}

#define MOE_R8(r, o) "=r"(r[o]), "=r"(r[o + 1]), "=r"(r[o + 2]), "=r"(r[o + 3]), "=r"(r[o + 4]), "=r"(r[o + 5]), \
                     "=r"(r[o + 6]), "=r"(r[o + 7])
#define MOE_I8(r, o) "r"(r[o]), "r"(r[o + 1]), "r"(r[o + 2]), "r"(r[o + 3]), "r"(r[o + 4]), "r"(r[o + 5]), \
                     "r"(r[o + 6]), "r"(r[o + 7])

// 32 columns of this warp's 32 lanes (the load still has to be waited for)
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t *r)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
                 "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : MOE_R8(r, 0), MOE_R8(r, 8), MOE_R8(r, 16), MOE_R8(r, 24)
                 : "r"(taddr));
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
                 MOE_I8(r, 0), MOE_I8(r, 8), MOE_I8(r, 16), MOE_I8(r, 24)
                 : "memory");
}

__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tma_4d(void *dst, const CUtensorMap *map, int x, int y, int z, int w, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
        "%5}], [%6];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
        : "memory");
}

// Bounded waits (gemm_common.cuh) without calls: a function's registers are the launch's, which the warps here have
// shared out anew.
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity, volatile int *abort_flag, int *err)
{
    if (mbar_try_wait(bar, parity))
        return true;
    const uint64_t t0 = global_ns();
#pragma unroll 1
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait(bar, parity))
            return true;
        if ((i & 7u) == 0) {
            if (*abort_flag)
                return false;
            if (global_ns() - t0 > WAIT_LIMIT_NS) {
                atomicCAS(err, 0, DEV_ERR_WAIT_TIMEOUT);
                *abort_flag = 1;
                return false;
            }
        }
    }
}

__device__ __forceinline__ bool wait_for_warp(uint64_t *bar, uint32_t parity, volatile int *abort_flag, int *err)
{
    return __all_sync(0xffffffffu, wait_for(bar, parity, abort_flag, err)) != 0;
}

__device__ __forceinline__ void drain(uint64_t *bar, uint32_t parity)
{
    const uint64_t t0 = global_ns();
#pragma unroll 1
    while (!mbar_try_wait(bar, parity) && global_ns() - t0 <= WAIT_LIMIT_NS) {
    }
}

// ---------------------------------------------------------------- which rows

struct Span {
    int start, len;
};

__device__ __forceinline__ Span sequence(const PromptArgs &a, int b)
{
    const int s = min(max(__ldcg(a.offsets + b), 0), a.T), e = min(max(__ldcg(a.offsets + b + 1), s), a.T);
    return {s, e - s};
}

// One piece of work: the two tiles from token tok0 (within the sequence) on, of a key head; len == 0: no more
struct Item {
    int start, len, tok0, kvh;
};

// The list of all items holds, from the highest level down, the level-th item of every sequence that has one: the
// rows that see most keys come first.  One warp walks it for its CTA.
struct Walk {
    static constexpr int KEPT = 4;  // sequences of a lane whose items it keeps
    int kept[KEPT], starts[KEPT], lens[KEPT];
    int level, here, over;          // the level it is at; items at this level and above, and above it
    int b0, seen;                   // sequences looked at, and those of them that have an item at this level

    __device__ __forceinline__ int items(const PromptArgs &a, int b) const
    {
        const int per = 2 * a.tile_tokens;
        return b < a.n_seqs ? (sequence(a, b).len + per - 1) / per : 0;
    }

    // (Cut where no call with ascending offsets comes: T and n_seqs allow less than MOST items of a key head.)
    __device__ __forceinline__ int above(const PromptArgs &a, int at_level, int lane) const
    {
        constexpr int MOST = 1 << 25;
        int s = 0;
#pragma unroll
        for (int i = 0; i < KEPT; ++i)
            s += max(0, kept[i] - at_level);
        for (int b = lane + 32 * KEPT; b < a.n_seqs; b += 32)
            s = min(MOST, s + max(0, items(a, b) - at_level));
        return (int)min(0x7FFFFFFFll, (long long)__reduce_add_sync(0xffffffffu, min(MOST, s)) * a.kv);
    }

    __device__ __forceinline__ void begin(const PromptArgs &a, int lane)
    {
#pragma unroll
        for (int i = 0; i < KEPT; ++i) {
            const Span q = lane + 32 * i < a.n_seqs ? sequence(a, lane + 32 * i) : Span{0, 0};
            starts[i] = q.start;
            lens[i] = q.len;
            kept[i] = (q.len + 2 * a.tile_tokens - 1) / (2 * a.tile_tokens);
        }
        level = a.T / (2 * a.tile_tokens) + 1;
        here = over = b0 = seen = 0;
    }

    // Item i of the list; i grows from call to call.  (Offsets that do not ascend may name more items than the rows have
    // room for: those are left out.)
    __device__ __forceinline__ Item at(const PromptArgs &a, int i, int lane)
    {
        if (i >= a.max_items)
            return {0, 0, 0, 0};
        if (i >= here) {  // down in steps that double, then between the last two: above(lo) > i >= above(hi)
            int hi = level, lo = level, n = here;
            for (int step = 1; n <= i; step *= 2) {
                if (lo == 0)
                    return {0, 0, 0, 0};
                hi = lo;
                over = n;
                lo = max(0, hi - step);
                n = above(a, lo, lane);
            }
            here = n;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                n = above(a, mid, lane);
                if (n > i) {
                    lo = mid;
                    here = n;
                } else {
                    hi = mid;
                    over = n;
                }
            }
            level = lo;
            b0 = seen = 0;
        }
        const int rank = (i - over) / a.kv, kvh = (i - over) - rank * a.kv;
        // the rank-th sequence with more than `level` items; ranks of a level grow from call to call
        for (;; b0 += 32) {
            if (b0 >= a.n_seqs)
                break;
            const int k = b0 >> 5;
            int n = 0;
#pragma unroll
            for (int j = 0; j < KEPT; ++j)
                n = k == j ? kept[j] : n;
            if (k >= KEPT)
                n = items(a, b0 + lane);
            uint32_t with = __ballot_sync(0xffffffffu, n > level);
            const int count = __popc(with);
            if (count > 0 && rank < seen + count) {
                for (int j = rank - seen; j > 0; --j)
                    with &= with - 1;
                const int from = __ffs(with) - 1;
                Span q = {0, 0};
#pragma unroll
                for (int j = 0; j < KEPT; ++j)
                    q = k == j ? Span{starts[j], lens[j]} : q;
                q.start = __shfl_sync(0xffffffffu, q.start, from);
                q.len = __shfl_sync(0xffffffffu, q.len, from);
                if (k >= KEPT)
                    q = sequence(a, b0 + from);
                return {q.start, q.len, level * 2 * a.tile_tokens, kvh};
            }
            seen += count;
        }
        return {0, 0, 0, 0};  // (not reached: offsets do not change during the call)
    }
};

// 32 bytes of a row
__device__ __forceinline__ void st256(uint16_t *p, const uint32_t *w)
{
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

__device__ __forceinline__ void st128x2(uint16_t *p, const uint32_t *w)
{
    reinterpret_cast<uint4 *>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4 *>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

// Adds to a row's sums what is not finite among the n values of a place in v and on, per value: what the sum over all
// of them would be (a probability is above 0).
template <int W> __device__ __forceinline__ void add_cleared(const uint16_t *v, long long ld, int n, uint32_t (&o)[W])
{
#pragma unroll 1
    for (int r = 0; r < n; ++r) {
#pragma unroll
        for (int c = 0; c < W; c += 2) {
            const uint32_t w = __ldcg(reinterpret_cast<const uint32_t *>(v + r * ld + c));
            const float x = __uint_as_float(w << 16), y = __uint_as_float(w & 0xFFFF0000u);
            o[c] = isfinite(x) ? o[c] : __float_as_uint(__uint_as_float(o[c]) + x);
            o[c + 1] = isfinite(y) ? o[c + 1] : __float_as_uint(__uint_as_float(o[c + 1]) + y);
        }
    }
}

// Key tiles of an item's two row tiles; those from `masked` on hold keys that some row must not see.
struct Tiles {
    int n0, n1, n, masked;
};

__device__ __forceinline__ Tiles tiles_of(const PromptArgs &a, const Item &item)
{
    const int last = item.len - 1, second = item.tok0 + a.tile_tokens;
    Tiles t;
    t.n0 = min(last, second - 1) / BN + 1;
    t.n1 = second > last ? 0 : min(last, second + a.tile_tokens - 1) / BN + 1;
    t.n = max(t.n0, t.n1);
    t.masked = item.tok0 / BN;
    return t;
}

// ---------------------------------------------------------------- kernel

template <int D>
__global__ void __launch_bounds__(THREADS, 1)
    prompt_kernel(const __grid_constant__ PromptArgs a, const __grid_constant__ CUtensorMap map_q,
                  const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v)
{
    using G = PGeo<D>;
    extern __shared__ uint8_t smem_dyn[];
    __shared__ Item items[2];
    __shared__ uint32_t tmem_word;
    __shared__ int abort_word, odd_word;  // odd: a value that is not finite has been cleared, in this item or an earlier
    volatile int *abort_flag = &abort_word;
    uint8_t *smem = smem_dyn + ((1024u - (smem_addr(smem_dyn) & 1023u)) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + G::BAR_OFF), *empty = full + G::SLOTS;
    uint64_t *v_land = empty + G::SLOTS, *v_clear = v_land + G::SLOTS, *s_full = v_clear + G::SLOTS, *p_full = s_full + 2;
    uint64_t *s_free = p_full + 2, *o_full = s_free + 2, *q_full = o_full + 2, *q_empty = q_full + 1, *item_full = q_empty + 1;
    uint64_t *item_empty = item_full + 2, *end_bar = item_empty + 2;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < G::SLOTS; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
            mbar_init(&v_land[i], 1);
            mbar_init(&v_clear[i], GUARDS);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&s_full[t], 1);
            mbar_init(&p_full[t], 4);
            mbar_init(&s_free[t], 4);
            mbar_init(&o_full[t], 1);
            mbar_init(&item_full[t], 1);
            mbar_init(&item_empty[t], THREADS / 32 - 1);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        mbar_init(end_bar, 1);
        abort_word = odd_word = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async();
    }
    // (a kernel that started before this one's end may hold tensor memory while it waits for that end: this one takes
    // its own only when nothing is left before it, and lets the next one start only then)
    overlap_wait();
    if (warp == WARP_MMA) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_word)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    overlap_trigger();
    const uint32_t tmem = tmem_word;

    // the CTA's next item, for every warp but the loader's: i counts them
    auto next_item = [&](int i, Item &item) {
        if (!wait_for_warp(&item_full[i & 1], (i >> 1) & 1, abort_flag, a.err))
            return false;
        item = items[i & 1];
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&item_empty[i & 1]);
        return item.len > 0;
    };

    if (warp == WARP_LOAD) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(OTHER_REGS));
        // ------------------------------------------------------ items, and tiles -> shared memory
        // Items go to the CTAs forth and back, so that none has the longest of every round.  K0 V0 K1 V1 ... of an item;
        // the values of masked tiles land on another barrier of their slot, where the guards wait for them.  Everyone who
        // waits for a slot's barrier so waits for each of its phases, and none comes before the slot was free again: no
        // phase can pass unseen.
        Walk walk;
        walk.begin(a, lane);
        int slot = 0;
        uint32_t ph = 0, slot_parity = 0, land_parity = 0, armed = 0, armed_land = 0;
        bool ok = true;
        const int ctas = (int)gridDim.x, cta = (int)blockIdx.x;
        auto load_q = [&](const Item &item, const Tiles &tl) {
            if (lane == 0) {
                const int rows = a.group * a.tile_tokens, both = tl.n1 > 0 ? 2 : 1;
                mbar_arrive_expect_tx(q_full, both * rows * D * 2);
                for (int t = 0; t < both; ++t)
                    for (int h = 0; h < D / 64; ++h)
                        tma_4d(smem + t * G::TILE_B + h * (BM * 128), &map_q, 0, item.kvh * a.group,
                               item.start + item.tok0 + t * a.tile_tokens, h, q_full);
            }
        };
        for (int i = 0; ok; ++i) {
            const Item item = walk.at(a, i & 1 ? (i + 1) * ctas - 1 - cta : i * ctas + cta, lane);
            if (!(ok = wait_for_warp(&item_empty[i & 1], ((i >> 1) & 1) ^ 1, abort_flag, a.err)))
                break;
            if (lane == 0) {
                items[i & 1] = item;
                mbar_arrive(&item_full[i & 1]);
            }
            if (item.len == 0)
                break;
            const Tiles tl = tiles_of(a, item);
            if (i == 0)
                load_q(item, tl);
            for (int it = 0; it < 2 * tl.n; ++it) {
                const int j = it >> 1;
                const bool is_v = it & 1;
                if (!(ok = wait_for_warp(&empty[slot], ph ^ 1, abort_flag, a.err)))
                    break;
                const bool land = is_v && j >= tl.masked;
                if (lane == 0) {
                    uint64_t *bar = land ? &v_land[slot] : &full[slot];
                    mbar_arrive_expect_tx(bar, G::TILE_B);
                    tma_4d(smem + G::RING_OFF + slot * G::TILE_B, is_v ? &map_v : &map_k, 0, item.kvh, item.start + j * BN,
                           0, bar);
                }
                if (land) {
                    land_parity ^= 1u << slot;
                    armed_land |= 1u << slot;
                } else {
                    slot_parity ^= 1u << slot;
                    armed |= 1u << slot;
                }
                if (++slot == G::SLOTS) {
                    slot = 0;
                    ph ^= 1;
                }
                if (it == 1 && i > 0) {  // (the queries' place is free later than the first tiles')
                    if (!(ok = wait_for_warp(q_empty, (i & 1) ^ 1, abort_flag, a.err)))
                        break;
                    load_q(item, tl);
                }
            }
        }
        // every copy has landed before the CTA ends (at once on the normal path, where the MMAs have read them; bounded)
        if (lane == 0 && !ok) {
            for (int i = 0; i < G::SLOTS; ++i)
                if (armed >> i & 1)
                    drain(&full[i], (slot_parity >> i & 1) ^ 1);
            for (int i = 0; i < G::SLOTS; ++i)
                if (armed_land >> i & 1)
                    drain(&v_land[i], (land_parity >> i & 1) ^ 1);
            drain(q_full, 0);
            drain(q_full, 1);
        }
        __syncwarp();
    } else if (warp >= WARP_GUARD) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(OTHER_REGS));
        // ------------------------------------------------------ values that no row, or not every row, may see
        Item item;
        int slot = 0;              // of the item's first key tile
        uint32_t land_parity = 0;
        for (int i = 0; next_item(i, item); ++i) {
            const Tiles tl = tiles_of(a, item);
            bool ok = true;
            for (int j = tl.masked; j < tl.n; ++j) {
                const int at = (slot + 2 * j + 1) % G::SLOTS;
                if (!(ok = wait_for_warp(&v_land[at], land_parity >> at & 1, abort_flag, a.err)))
                    break;
                land_parity ^= 1u << at;
                uint8_t *tile = smem + G::RING_OFF + at * G::TILE_B;
                const int held = item.len - j * BN;  // rows of the tile within the sequence
                const int me = (warp - WARP_GUARD) * 32 + lane;
                bool odd = false;
                // (rows past the end: a sequence's last tile alone has any)
                for (int h = 0; h < D / 64; ++h)
                    for (int c = max(0, held) * 8 + me; c < BN * 8; c += GUARDS * 32)
                        reinterpret_cast<uint4 *>(tile)[h * BN * 8 + c] = make_uint4(0, 0, 0, 0);
                __syncwarp();  // (both guards may write the same zeros: what one reads as it was it leaves)
#pragma unroll 1
                for (int c = me; c < G::TILE_B / 16; c += 8 * GUARDS * 32) {
                    uint4 v[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        v[k] = reinterpret_cast<const uint4 *>(tile)[c + k * GUARDS * 32];
                    uint32_t any = 0;  // an exponent of ones carries into the sign's place
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        any |= ((v[k].x & 0x7F807F80u) + 0x00800080u) | ((v[k].y & 0x7F807F80u) + 0x00800080u) |
                               ((v[k].z & 0x7F807F80u) + 0x00800080u) | ((v[k].w & 0x7F807F80u) + 0x00800080u);
                    if (!(any & 0x80008000u))
                        continue;
#pragma unroll 1
                    for (int k = 0; k < 8; ++k) {
                        uint32_t *w = reinterpret_cast<uint32_t *>(tile) + 4 * (c + k * GUARDS * 32);
                        if ((c + k * GUARDS * 32) / 8 % BN >= held)
                            continue;  // (already, or about to be, zeros)
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t x = w[i];
                            const uint32_t clear = ((x & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u) |
                                                   ((x & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u);
                            if (clear) {
                                w[i] = x & ~clear;
                                odd = true;
                            }
                        }
                    }
                }
                if (odd)
                    odd_word = 1;
                __threadfence_block();
                fence_proxy_async();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&v_clear[at]);
            }
            if (!ok)
                break;
            slot = (slot + 2 * tl.n) % G::SLOTS;
        }
        __syncwarp();
    } else if (warp == WARP_MMA) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(OTHER_REGS));
        // ------------------------------------------------------ MMAs: the warp runs the loop, one elected lane issues
        uint32_t elected;
        asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(elected));
        auto wait = [&](uint64_t *bar, uint32_t par) {
            return wait_for_warp(bar, par, abort_flag, a.err);
        };
        const uint64_t dq = desc_k(smem_addr(smem)), dk = desc_k(smem_addr(smem + G::RING_OFF));
        const uint64_t dv = desc_n(smem_addr(smem + G::RING_OFF));
        constexpr uint64_t TILE16 = G::TILE_B / 16, HALF16 = BM * 128 / 16;
        uint32_t slot_parity = 0, clear_parity = 0, p_parity = 0, s_parity = 3;
        int slot = 0;
        auto wait_slot = [&](int at) {
            if (!wait(&full[at], slot_parity >> at & 1))
                return false;
            slot_parity ^= 1u << at;
            return true;
        };
        auto scores = [&](int t, int at) {  // S of row tile t and the keys in the slot
            if (elected) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint64_t o = (k / 4) * HALF16 + (k % 4) * 2;
                    mma_ss(tmem + t * BN, dq + t * TILE16 + o, dk + at * TILE16 + o, instr_desc(BN, false), k > 0);
                }
                commit(&s_full[t]);
            }
            __syncwarp();
        };
        auto next_scores = [&](int t, int at) {  // with P apart: once the tile's rows have their last S in registers
            if (G::APART) {
                if (!wait(&s_free[t], s_parity >> t & 1))
                    return false;
                s_parity ^= 1u << t;
                fence_after();
            }
            scores(t, at);
            return true;
        };
        // The first tile's first S of an item, as soon as the queries and keys are there.  It comes before the last P of
        // the second tile of the item before: the two tiles' softmaxes keep to their turns from item to item.  (The
        // queries' place is free once the second tile's last S has been issued, a round earlier.)
        auto begin = [&](int i, int at) {
            if (!wait(q_full, i & 1) || !wait_slot(at))
                return false;
            fence_after();
            return next_scores(0, at);
        };
        Item item;
        bool ok = true, more = next_item(0, item);
        if (more)
            more = begin(0, 0);
        for (int i = 0; more; ++i) {
            const Tiles tl = tiles_of(a, item);
            more = false;
            // (P of the item before, where it lies in these columns, has its products before these in the queue)
            if (tl.n1 > 0 && !next_scores(1, slot))
                break;
            if (elected) {
                commit(&empty[slot]);
                if (tl.n == 1)
                    commit(q_empty);
            }
            __syncwarp();
            for (int j = 0; j < tl.n; ++j) {
                const int vs = slot + 1 < G::SLOTS ? slot + 1 : 0, ks = vs + 1 < G::SLOTS ? vs + 1 : 0;
                if (j >= tl.masked) {
                    if (!(ok = wait(&v_clear[vs], clear_parity >> vs & 1)))
                        break;
                    clear_parity ^= 1u << vs;
                } else if (!(ok = wait_slot(vs))) {
                    break;
                }
                if (j + 1 < tl.n && !(ok = wait_slot(ks)))
                    break;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int nt = t ? tl.n1 : tl.n0;
                    if (t == 1 && ok && j + 1 == tl.n && next_item(i + 1, item))
                        more = ok = begin(i + 1, ks);
                    if (j >= nt || !ok)
                        continue;
                    // (the first tile's P comes before the second's next S: the two tiles' softmaxes so run in turns)
                    if (G::APART && j + 1 < nt && !(ok = next_scores(t, ks)))
                        continue;
                    if (!(ok = wait(&p_full[t], p_parity >> t & 1)))
                        continue;
                    p_parity ^= 1u << t;
                    fence_after();
                    if (elected) {
#pragma unroll
                        for (int k = 0; k < BN / 16; ++k)
                            mma_ts(tmem + G::O_COL + t * D, tmem + G::P_COL + t * G::P_STEP + 8 * k, dv + vs * TILE16 + k * (16 * 128 / 16),
                                   instr_desc(D, true), j > 0 || k > 0);
                        if (G::APART || j + 1 == nt)
                            commit(&o_full[t]);
                    }
                    __syncwarp();
                    if (!G::APART && j + 1 < nt)
                        scores(t, ks);
                }
                if (!ok)
                    break;
                if (elected) {
                    commit(&empty[vs]);
                    if (j + 1 < tl.n)
                        commit(&empty[ks]);
                    if (j + 2 == tl.n)
                        commit(q_empty);
                }
                __syncwarp();
                slot = ks;  // (after the last tile: the next item's first)
            }
            more = more && ok;
        }
        // also after an abort: what was issued has completed before the tensor memory is freed
        if (elected) {
            commit(end_bar);
            drain(end_bar, 0);
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(SOFTMAX_REGS));
        // ------------------------------------------------------ softmax: a thread per row
        const int t = warp >> 2, row = (warp & 3) * 32 + lane, in_tile = row / a.group, head = row - in_tile * a.group;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + t * BN, to = tmem + lanes + G::O_COL + t * D;
        const uint32_t tp = tmem + lanes + G::P_COL + t * G::P_STEP;
        uint32_t s_parity = 0, o_parity = 0;
        Item item;
        for (int i = 0; next_item(i, item); ++i) {
            const Tiles tl = tiles_of(a, item);
            const int nt = t ? tl.n1 : tl.n0;
            if (nt == 0)
                continue;
            const int tok = item.tok0 + t * a.tile_tokens + in_tile;  // within the sequence
            const bool valid = in_tile < a.tile_tokens && tok < item.len;
            const int sees = valid ? tok + 1 : 0x40000000;  // keys that the row sees
            float m = -INFINITY, l = 0.f;                   // m: of scaled scores, the one in use
            bool ok = true;
            for (int j = 0; j < nt; ++j) {
                if (!(ok = wait_for_warp(&s_full[t], s_parity, abort_flag, a.err)))
                    break;
                s_parity ^= 1;
                fence_after();
                uint32_t s[BN];
#pragma unroll
                for (int c = 0; c < BN; c += 32)
                    tmem_ld32(ts + c, s + c);
                wait_ld();
                if (G::APART) {
                    fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&s_free[t]);
                }
                if (j >= tl.masked) {
                    const int vis = sees - j * BN;
#pragma unroll
                    for (int c = 0; c < BN; ++c)
                        s[c] = c < vis ? s[c] : 0xFF800000u;
                }
                const float mx = a.scale * row_max(s);
                if (G::APART && j > 0) {  // the product before is done: O may be touched and P overwritten (with S and P
                                          // in one place that a new S is there says so)
                    if (!(ok = wait_for_warp(&o_full[t], o_parity, abort_flag, a.err)))
                        break;
                    o_parity ^= 1;
                    fence_after();
                }
                const bool grown = mx > m + GROWTH && valid;
                if (j == 0) {
                    m = mx;
                } else if (__any_sync(0xffffffffu, grown)) {
                    const float next = grown ? mx : m, f = ex2(m - (next == -INFINITY ? 0.f : next));
                    m = next;
                    l *= f;
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        uint32_t o[32];
                        tmem_ld32(to + c, o);
                        wait_ld();
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                        tmem_st32(to + c, o);
                    }
                }
                const float base = m == -INFINITY ? 0.f : m;
                const uint64_t mul2 = pack2(a.scale, a.scale), base2 = pack2(-base, -base);
                uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
                for (int c = 0; c < BN; c += 64) {
                    uint32_t p[32];
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        const float2 x = unpack2(fma2(pack2(__uint_as_float(s[c + 2 * k]), __uint_as_float(s[c + 2 * k + 1])),
                                                      mul2, base2));
                        const float p0 = ex2(x.x), p1 = ex2(x.y);
                        sum[k & 3] = add2(sum[k & 3], pack2(p0, p1));
                        // Rounded to BF16 for the product (2^-8 of each at most, of random sign: errors of 0.0020 of
                        // the norm against 64 bits, 0.0016 without): v is BF16, and an MMA's operands share a type.
                        // What the rounding leaves, in a product of its own, would take the tensor pipe from 2,048 to
                        // 3,072 of a key tile's 2,900 cycles.  The sum is of the exact P: of the rounded ones it brought
                        // 0.0019 and cost two instructions a pair (8192 rows 676 -> 716 us).
                        p[k] = bf16_pair(p0, p1);
                    }
                    tmem_st32(tp + c / 2, p);
                }
                const float2 sums = unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
                l += sums.x + sums.y;
                wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&p_full[t]);
            }
            ok = ok && wait_for_warp(&o_full[t], o_parity, abort_flag, a.err);
            if (!ok)
                break;
            o_parity ^= 1;
            fence_after();
            const float inv = 1.f / l;
            const bool odd = *static_cast<volatile int *>(&odd_word) != 0;
            const long long at = item.start + tok;
            const bool wide = a.wide_out;
            uint16_t *out = a.out + at * a.out_ld + (long long)(item.kvh * a.group + head) * D;
            // (a loop: code that runs once an item is not in the instruction cache, and unrolled it takes longer to come
            // than to run)
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tmem_ld32(to + c, o);
                wait_ld();
                if (odd && valid)  // what the guards cleared, for the rows that see it
                    add_cleared<32>(a.v + (item.start + tl.masked * BN) * a.v_ld + (long long)item.kvh * D + c, a.v_ld,
                                    tok - tl.masked * BN + 1, o);
                uint32_t w[16];
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    w[k] = bf16_pair(__uint_as_float(o[2 * k]) * inv, __uint_as_float(o[2 * k + 1]) * inv);
                if (valid && wide) {
                    st256(out + c, w);
                    st256(out + c + 16, w + 8);
                } else if (valid) {
                    st128x2(out + c, w);
                    st128x2(out + c + 16, w + 8);
                }
            }
            fence_before();  // (the next item's first product into O waits for its P, which comes after this)
        }
    }
    __syncthreads();
    if (warp == WARP_MMA) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
    }
}

// ---------------------------------------------------------------- host side

MoeStatus bad(MoeStatus s, const char *msg) { return (MoeStatus)set_last_error(s, msg); }

// rows as {64 values, heads, rows, 64-value parts of a head}, boxes of {64, box_heads, box_rows, parts}
cudaError_t rows_map(CUtensorMap *m, const void *base, long long ld, int T, int heads, int D, int box_heads,
                     int box_rows, int box_parts)
{
    auto enc = tensor_map_encoder();
    if (!enc)
        return cudaErrorNotSupported;
    const cuuint64_t dims[4] = {64, (cuuint64_t)heads, (cuuint64_t)T, (cuuint64_t)(D / 64)};
    const cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)ld * 2, 128};
    const cuuint32_t box[4] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows, (cuuint32_t)box_parts};
    const cuuint32_t step[4] = {1, 1, 1, 1};
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, step,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D>
cudaError_t launch_prompt(PromptArgs &a, const void *q, long long q_ld, const void *k, long long k_ld,
                          cudaStream_t st)
{
    auto kern = prompt_kernel<D>;
    static std::atomic<int> attr_set[MAX_DEVICES];
    CUtensorMap mq, mk, mv;
    cudaError_t e = smem_limit_once(attr_set, (const void *)kern, PGeo<D>::SMEM);
    if (e == cudaSuccess)
        e = rows_map(&mq, q, q_ld, a.T, a.heads, D, a.group, a.tile_tokens, 1);
    if (e == cudaSuccess)
        e = rows_map(&mk, k, k_ld, a.T, a.kv, D, 1, BN, D / 64);
    if (e == cudaSuccess)
        e = rows_map(&mv, a.v, a.v_ld, a.T, a.kv, D, 1, BN, D / 64);
    if (e != cudaSuccess)
        return e;
    // a CTA per SM, or per item where there are fewer (at most: every sequence rounds up to whole items)
    const long long items = ((long long)a.T / (2 * a.tile_tokens) + a.n_seqs) * a.kv;
    const long long grid = items < sm_count() ? items : sm_count();
    a.max_items = (int)items;
    return launch_overlapped(kern, (unsigned)grid, THREADS, PGeo<D>::SMEM, 1, st, a, mq, mk, mv);
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" MoeStatus moe_attention_prompt(const void *q, long long q_ld, const void *k, long long k_ld, const void *v,
                                          long long v_ld, int T, const int32_t *offsets, int n_seqs, int n_heads,
                                          int n_kv_heads, int head_dim, float scale, void *out, long long out_ld,
                                          void *cuda_stream)
{
    char msg[160];
    const int D = head_dim;
    if (T < 0 || T > (1 << 24) || n_seqs < 0 || n_seqs > 65536) {
        snprintf(msg, sizeof msg, "T = %d or n_seqs = %d out of range [0, 2^24], [0, 65536]", T, n_seqs);
        return bad(MOE_EINVAL, msg);
    }
    if (D != 64 && D != 128) {
        snprintf(msg, sizeof msg, "moe_attention_prompt: head_dim (%d) must be 64 or 128", D);
        return bad(MOE_EDIMS, msg);
    }
    if (n_heads < 1 || n_heads > ATTN_MAX_HEADS || n_kv_heads < 1 || n_heads % n_kv_heads || n_heads / n_kv_heads > 64) {
        snprintf(msg, sizeof msg, "n_heads (%d) must be 1 to 64 times n_kv_heads (%d) and at most %d", n_heads,
                 n_kv_heads, ATTN_MAX_HEADS);
        return bad(MOE_EINVAL, msg);
    }
    if (!(scale > 0.f) || !isfinite(scale * 1.4427f))
        return bad(MOE_EINVAL, "moe_attention_prompt: scale must be finite and above 0");
    if (T == 0 || n_seqs == 0)
        return MOE_OK;
    if (!q || !k || !v || !offsets || !out)
        return bad(MOE_EINVAL, "moe_attention_prompt: NULL q, k, v, offsets or out");
    const long long wq = (long long)n_heads * D, wk = (long long)n_kv_heads * D;
    if (q_ld < wq || out_ld < wq || k_ld < wk || v_ld < wk)
        return bad(MOE_EINVAL, "moe_attention_prompt: a row stride is below the row's values");
    if (!rows_16b(q, q_ld) || !rows_16b(k, k_ld) || !rows_16b(v, v_ld) || !rows_16b(out, out_ld) ||
        (uintptr_t)offsets % 4)
        return bad(MOE_EINVAL, "moe_attention_prompt: rows must start on 16-byte boundaries, offsets on 4-byte ones");
    PromptArgs a{};
    cudaError_t e = attention_error_flag(&a.err);
    if (e == cudaSuccess) {
        a.offsets = offsets;
        a.n_seqs = n_seqs;
        a.T = T;
        a.heads = n_heads;
        a.kv = n_kv_heads;
        a.group = n_heads / n_kv_heads;
        a.tile_tokens = BM / a.group;
        a.v = static_cast<const uint16_t *>(v);
        a.v_ld = v_ld;
        a.scale = scale * 1.44269504088896340736f;
        a.out = static_cast<uint16_t *>(out);
        a.out_ld = out_ld;
        a.wide_out = (uintptr_t)out % 32 == 0 && out_ld % 16 == 0;
        cudaStream_t st = (cudaStream_t)cuda_stream;
        e = D == 128 ? launch_prompt<128>(a, q, q_ld, k, k_ld, st) : launch_prompt<64>(a, q, q_ld, k, k_ld, st);
    }
    if (e != cudaSuccess) {
        snprintf(msg, sizeof msg, "prompt attention launch: %s", cudaGetErrorString(e));
        return bad(MOE_ECUDA, msg);
    }
    return MOE_OK;
}
