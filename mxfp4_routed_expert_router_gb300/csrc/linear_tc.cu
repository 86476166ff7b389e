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
// BF16 rows with BF16 operands, else FP16 rows x * 2^-e (a power of two per
// token) that a first kernel writes.
//
// A CTA computes one tile (128 rows x up to 128 tokens x its K range) and two CTAs
// share an SM (half of its tensor memory each), so that the hand-offs, the first
// loads and the epilogue of one overlap the MMAs of the other.  A cluster of 1, 2,
// 4 or 8 CTAs splits K; its partial tiles meet in shared memory and each rank
// finishes a share of the tokens, in a fixed order.  Warps: 0 loads tiles and
// prefetches weight chunks into L2, 1 issues the MMAs, 2-5 decode and then finish
// the tile.  Every mbarrier wait is bounded (gemm_common.cuh).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gemm_common.cuh"
#include "linear_internal.cuh"
#include "mx_decode.cuh"

namespace moe {

namespace {

using namespace gemm;

constexpr int N_WARPS = 6, THREADS = N_WARPS * 32;
constexpr int WARP_LOAD = 0, WARP_MMA = 1;  // 2-5: decode
constexpr int NMAX = 128;             // tokens of a tile
constexpr int A_STAGES = 2;           // A ring (tensor memory)
constexpr int A_SLOT_COLS = 64;       // 128 16-bit values per lane
constexpr int TMEM_COLS = 256;        // half of the SM's: accumulator and A ring
static_assert(NMAX + A_STAGES * A_SLOT_COLS <= TMEM_COLS, "tensor memory");
constexpr int SLICE_BYTES = NMAX * HALF_K * 2;           // 16 KB: 128 token rows x 64 values, one swizzled tile
constexpr int A_TILE_BYTES = TILE_ROWS * HALF_K * 2;     // BF16 weights: 16 KB
constexpr int RING_BYTES = 96 * 1024;
constexpr int RING_MAX = 6;
constexpr int BAR_OFF = RING_BYTES;
constexpr int N_BARS = 2 * RING_MAX + 2 * A_STAGES + 1;
constexpr int MISC_OFF = BAR_OFF + N_BARS * 8;
constexpr int TSC_OFF = MISC_OFF + 16;                   // token scales of the tile
constexpr int SMEM_BYTES = TSC_OFF + NMAX * 4 + 1024;    // + alignment slack
static_assert(2 * (SMEM_BYTES + 1024) <= 228 * 1024, "two CTAs per SM");
static_assert(NMAX * TILE_ROWS * 4 <= RING_BYTES, "a partial tile fits in the ring");
constexpr int PF_CHUNKS = 8;          // weight chunks prefetched into L2 ahead of the stage being loaded

struct Args {
    const uint8_t *w;
    const uint8_t *row_base;  // FP16 operands: power of two (+ 127) of each row
    const float *xscale;      // FP16 operands: power of two of each token
    int N, T, kchunks, chunk_bytes;
    int tile_tokens;          // tokens of a tile (a multiple of 16, at most NMAX), rows of a TMA box of B
    int ttiles;
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
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t acc = k ? 1u : acc0;
        if (AS)
            asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                         " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
                         "l"(a_desc + 2 * k), "l"(b + 2 * k), "r"(idesc), "r"(acc)
                         : "memory");
        else
            asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                         " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
                         "r"(a_tmem + 8 * k), "l"(b + 2 * k), "r"(idesc), "r"(acc)
                         : "memory");
    }
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

template <int OP, int WFMT>
__global__ void __launch_bounds__(THREADS, 2)
    linear_tc_kernel(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap map_b,
                     const __grid_constant__ CUtensorMap map_a)
{
    constexpr bool AS = WFMT == FMT_BF16;                            // A by TMA into shared memory
    constexpr int KST = (AS || OP == LIN_I4) ? HALF_K : CHUNK_K;     // K values per stage
    constexpr int NSL = KST / HALF_K;                                // 64-wide slices per stage
    constexpr int NBLK = KST / 32;
    constexpr int STAGE_BYTES = NSL * SLICE_BYTES + (AS ? A_TILE_BYTES : 0);
    constexpr int RING = RING_BYTES / STAGE_BYTES;                   // 3 of 32 KB, or 6 of 16 KB
    static_assert(RING >= 3 && RING <= RING_MAX, "ring");
    extern __shared__ uint8_t smem_dyn[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
    uint64_t *b_full = reinterpret_cast<uint64_t *>(smem + BAR_OFF), *b_empty = b_full + RING_MAX;
    uint64_t *a_full = b_empty + RING_MAX, *a_empty = a_full + A_STAGES, *acc_full = a_empty + A_STAGES;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + MISC_OFF);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + MISC_OFF + 4);
    float *tsc = reinterpret_cast<float *>(smem + TSC_OFF);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t crank, csize;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(crank));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(csize));
    const int item = blockIdx.x / csize, rt = item / a.ttiles, tt = item - rt * a.ttiles;
    const int tok0 = tt * a.tile_tokens, nvalid = min(a.tile_tokens, a.T - tok0);
    const int n_mma = (nvalid + 15) & ~15;
    const int c0 = (int)((long long)a.kchunks * crank / csize), c1 = (int)((long long)a.kchunks * (crank + 1) / csize);
    const int nst = (c1 - c0) * (CHUNK_K / KST);
    const uint8_t *wsrc = a.w + ((size_t)rt * a.kchunks + c0) * (size_t)a.chunk_bytes;

    if (tid == 0) {
        for (int i = 0; i < RING; ++i) {
            mbar_init(&b_full[i], 1);
            mbar_init(&b_empty[i], 1);
        }
        for (int i = 0; i < A_STAGES; ++i) {
            mbar_init(&a_full[i], 4);
            mbar_init(&a_empty[i], 1);
        }
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
    if (OP != LIN_BF16)
        for (int i = tid; i < nvalid; i += THREADS)
            tsc[i] = __ldg(a.xscale + tok0 + i);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tmem_a = tmem + NMAX;

    if (warp == WARP_LOAD) {
        // ---------------------------------------------------------- tiles -> ring
        int pf = 0;
        auto prefetch = [&]() {
            if (pf < c1 - c0 && lane == 0 && !AS)
                asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(wsrc + (size_t)pf * a.chunk_bytes),
                             "r"((uint32_t)a.chunk_bytes)
                             : "memory");
            ++pf;
        };
        for (int i = 0; i < PF_CHUNKS; ++i)
            prefetch();
        const uint32_t bytes = (uint32_t)(NSL * a.tile_tokens * HALF_K * 2 + (AS ? A_TILE_BYTES : 0));
        int st = 0;
        for (; st < nst; ++st) {
            const int slot = st % RING;
            if (!mbar_wait_sleep_warp(&b_empty[slot], ((st / RING) & 1) ^ 1, abort_flag, a.err, lane))
                break;
            if (KST == CHUNK_K || (st & 1) == 0)
                prefetch();
            if (lane == 0) {
                uint8_t *dst = smem + slot * STAGE_BYTES;
                const int k = c0 * CHUNK_K + st * KST;
                mbar_arrive_expect_tx(&b_full[slot], bytes);
#pragma unroll
                for (int s = 0; s < NSL; ++s)
                    tma_2d(dst + s * SLICE_BYTES, &map_b, k + s * HALF_K, tok0, &b_full[slot]);
                if (AS)  // the store seen as [row tiles * chunks * 2 halves * 128][64]
                    tma_2d(dst + NSL * SLICE_BYTES, &map_a, 0, ((rt * a.kchunks + c0) * 2 + st) * TILE_ROWS,
                           &b_full[slot]);
            }
        }
        // every copy of an armed stage has landed before the CTA goes on (at once
        // on the normal path; bounded after an abort)
        if (lane == 0)
            for (int s = st > RING ? st - RING : 0; s < st; ++s)
                mbar_drain(&b_full[s % RING], (s / RING) & 1);
        __syncwarp();
    } else if (warp == WARP_MMA) {
        // ---------------------------------------------------------- MMAs (lane 0)
        if (lane == 0) {
            const uint64_t desc0 = sw128(smem_addr(smem));
            const uint32_t idesc = instr_desc(OP == LIN_BF16, n_mma);
            for (int st = 0; st < nst; ++st) {
                const int bs = st % RING, as = st % A_STAGES;
                // a_full comes after the stage's B tiles too: its decoders wait for both
                if (!(AS ? mbar_wait(&b_full[bs], (st / RING) & 1, abort_flag, a.err)
                         : mbar_wait(&a_full[as], (st / A_STAGES) & 1, abort_flag, a.err)))
                    break;
                fence_after();
                const uint64_t bd = desc0 + (uint64_t)((bs * STAGE_BYTES) >> 4);
                const uint32_t at = tmem_a + as * A_SLOT_COLS;
                if (AS) {
                    mma64<true>(tmem, 0, bd + (uint64_t)((NSL * SLICE_BYTES) >> 4), bd, idesc, st);
                } else if (OP == LIN_I4) {
                    mma64<false>(tmem, at, 0, bd, idesc, st);
                    mma64<false>(tmem, at + 32, 0, bd, idesc, 1u);
                } else {
#pragma unroll
                    for (int s = 0; s < NSL; ++s)
                        mma64<false>(tmem, at + 32 * s, 0, bd + (uint64_t)((s * SLICE_BYTES) >> 4), idesc,
                                     st > 0 || s > 0);
                }
                commit(&b_empty[bs]);
                if (!AS)
                    commit(&a_empty[as]);
            }
            // also after an abort: what was issued has completed before the tensor
            // memory is freed and the ring reused
            commit(acc_full);
            mbar_drain(acc_full, 0);
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------- decode
        const int q = warp & 3, r = 32 * q + lane;  // lane quadrant; row of the tile
        const uint32_t tlane = (uint32_t)(32 * q) << 16;
        bool ok = true;
        if (!AS) {
            const int rb = OP == LIN_BF16 ? 127 : (int)__ldg(a.row_base + rt * TILE_ROWS + r);
            uint4 code[NBLK];
            uint32_t sc[NBLK];
            auto fetch = [&](int st) {
                const uint8_t *ch = wsrc + (size_t)(st * KST / CHUNK_K) * a.chunk_bytes;
                const int b0 = KST == CHUNK_K ? 0 : 2 * (st & 1);
#pragma unroll
                for (int b = 0; b < NBLK; ++b) {
                    const int blk = b0 + b;
                    if (OP == LIN_I4) {
                        code[b] = __ldg(reinterpret_cast<const uint4 *>(ch + (blk * TILE_ROWS + r) * 16));
                        sc[b] = (uint32_t)__ldg(reinterpret_cast<const uint16_t *>(ch + CHUNK_MX_CODE_BYTES) +
                                                blk * TILE_ROWS + r) |
                                (uint32_t)__ldg(ch + CHUNK_MX_CODE_BYTES + CHUNK_I4_SCALE_BYTES + blk * TILE_ROWS + r)
                                    << 16;
                    } else if (OP == LIN_F16) {
                        code[b] = __ldg(reinterpret_cast<const uint4 *>(ch + (blk * TILE_ROWS + r) * 16));
                        sc[b] = __ldg(ch + CHUNK_MX_CODE_BYTES + blk * TILE_ROWS + r);
                    } else {
                        code[b] = __ldg(reinterpret_cast<const uint4 *>(ch + (blk >> 1) * (CHUNK_MX_CODE_BYTES / 2) +
                                                                        r * 32 + (blk & 1) * 16));
                        sc[b] = __ldg(ch + CHUNK_MX_CODE_BYTES + r * 4 + blk);
                    }
                }
            };
            if (nst > 0)
                fetch(0);
            for (int st = 0; st < nst; ++st) {
                const int slot = st % A_STAGES;
                if (!(ok = mbar_wait_warp(&a_empty[slot], ((st / A_STAGES) & 1) ^ 1, abort_flag, a.err, lane)))
                    break;
                fence_after();
                const uint32_t dst = tmem_a + tlane + slot * A_SLOT_COLS;
#pragma unroll
                for (int b = 0; b < NBLK; ++b) {
                    const uint32_t w[4] = {code[b].x, code[b].y, code[b].z, code[b].w};
                    uint32_t o[16];
                    if (OP == LIN_I4) {
                        // relative to the row's base (the scale then lies below 2^12)
                        const float sf = __half2float(__ushort_as_half((unsigned short)(sc[b] & 0xFFFFu))) *
                                         __int_as_float((254 - rb) << 23);
                        const uint32_t s2 = (uint32_t)__half_as_ushort(__float2half_rn(sf)) * 0x10001u;
                        const uint32_t zz = (0x6400u + (sc[b] >> 16)) * 0x10001u;
                        uint32_t lo[16];
#pragma unroll
                        for (int c = 0; c < 4; ++c)
#pragma unroll
                            for (int p = 0; p < 4; ++p)
                                decode_i4(w[c] >> (4 * p), zz, s2, o[4 * c + p], lo[4 * c + p]);
                        tmem_st16(dst + 32 + b * 16, lo);
                    } else if (OP == LIN_F16) {
                        int d = (int)sc[b] - rb;
                        d = d < -24 ? -24 : (d > 0 ? 0 : d);  // (blocks past K, whose codes are 0)
                        const uint32_t s2 = f16x2_pow2(d);
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            decode_e2m1(w[c], s2, o + 4 * c);
                    } else {
                        const uint32_t s2 = e8m0_to_bf16x2(sc[b]);
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            decode_word(w[c], s2, o + 4 * c);
                    }
                    tmem_st16(dst + b * 16, o);
                }
                if (st + 1 < nst)
                    fetch(st + 1);
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                fence_before();
                if (!(ok = mbar_wait_warp(&b_full[st % RING], (st / RING) & 1, abort_flag, a.err, lane)))
                    break;
                if (lane == 0)
                    mbar_arrive(&a_full[slot]);
            }
        }
        // ---------------------------------------------------------- the tile's sums
        if (ok && mbar_wait_sleep_warp(acc_full, 0, abort_flag, a.err, lane)) {
            fence_after();
            const int n = rt * TILE_ROWS + r;
            const float wsc =
                OP == LIN_BF16 ? 1.f : ldexpf(1.f, (int)__ldg(a.row_base + rt * TILE_ROWS + r) - 127);
            float *part = reinterpret_cast<float *>(smem);  // [token][128]: the ring is free
            for (int c = 0; c < n_mma; c += 16) {
                float v[16];
                if (nst > 0)
                    tmem_ld16(tmem + tlane + c, v);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    if (c + j >= nvalid)
                        continue;
                    const float f = nst > 0 ? v[j] * wsc : 0.f;
                    if (csize > 1) {
                        part[(c + j) * TILE_ROWS + r] = f;
                    } else if (n < a.N) {
                        const float o = OP == LIN_BF16 ? f : f * tsc[c + j];
                        const long long at = (long long)(tok0 + c + j) * a.y_ld + n;
                        if (a.y_f32) {
                            float *y = static_cast<float *>(a.y) + at;
                            *y = a.accumulate ? *y + o : o;
                        } else {
                            static_cast<__nv_bfloat16 *>(a.y)[at] = __float2bfloat16_rn(o);
                        }
                    }
                }
            }
        }
        fence_before();
    }

    __syncwarp();
    if (csize > 1) {
        cluster_sync();
        // rank r finishes tokens r, r + csize, ... of the tile: a warp per token, four rows a lane
        if (!*abort_flag) {
            const uint32_t part = smem_addr(smem);
            for (int t = crank + csize * warp; t < nvalid; t += csize * N_WARPS) {
                float s[4] = {0.f, 0.f, 0.f, 0.f};
                const uint32_t local = part + (t * TILE_ROWS + lane * 4) * 4;
                for (uint32_t rk = 0; rk < csize; ++rk) {
                    uint32_t remote;
                    float4 f;
                    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rk));
                    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                                 : "=f"(f.x), "=f"(f.y), "=f"(f.z), "=f"(f.w)
                                 : "r"(remote));
                    s[0] += f.x, s[1] += f.y, s[2] += f.z, s[3] += f.w;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int n = rt * TILE_ROWS + lane * 4 + j;
                    const float o = OP == LIN_BF16 ? s[j] : s[j] * tsc[t];
                    if (n < a.N) {
                        const long long at = (long long)(tok0 + t) * a.y_ld + n;
                        if (a.y_f32) {
                            float *y = static_cast<float *>(a.y) + at;
                            *y = a.accumulate ? *y + o : o;
                        } else {
                            static_cast<__nv_bfloat16 *>(a.y)[at] = __float2bfloat16_rn(o);
                        }
                    }
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
__global__ void __launch_bounds__(256) linear_rows_kernel(const void *x, const uint8_t *xscales, long long x_ld,
                                                          int x_mx, int K, int bf16, uint16_t *out, float *scale)
{
    __shared__ uint32_t red[8];
    const long long t = blockIdx.x;
    auto load = [&](int v, float f[8]) {
        if (x_mx) {
            const uint2 u = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(x) + t * x_ld) + v);
            const int e = __ldg(xscales + t * (K / 32) + v / 4);
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
            const uint4 u = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(x) + t * x_ld) + v);
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
        for (int v = threadIdx.x; v < nv; v += 256) {
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
#pragma unroll
        for (int i = 0; i < 8; ++i)
            b = max(b, red[i]);
        const int e = max((int)(b >> 23) - 141, -126);
        mul = __int_as_float((127 - e) << 23);
        if (threadIdx.x == 0)
            scale[t] = __int_as_float((127 + e) << 23);
    }
    for (int v = threadIdx.x; v < nv; v += 256) {
        float f[8];
        uint32_t o[4];
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
        reinterpret_cast<uint4 *>(out + t * (long long)K)[v] = make_uint4(o[0], o[1], o[2], o[3]);
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
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM_BYTES;
    cfg.stream = st;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)cluster;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = cluster > 1;
    return cudaLaunchKernelEx(&cfg, kern, a, mb, ma);
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace

size_t linear_gemm_workspace(int K, int T) { return align256((size_t)T * K * 2) + align256((size_t)T * 4); }

cudaError_t launch_linear_gemm(const LinearGemm &g, cudaStream_t st)
{
    Args a{};
    a.w = g.w->base;
    a.row_base = g.w->row_base;
    a.N = g.N;
    a.T = g.T;
    a.kchunks = g.w->kchunks;
    a.chunk_bytes = g.w->chunk_bytes;
    a.ttiles = (g.T + NMAX - 1) / NMAX;
    a.tile_tokens = ((g.T + a.ttiles - 1) / a.ttiles + 15) & ~15;
    a.ttiles = (g.T + a.tile_tokens - 1) / a.tile_tokens;
    a.y = g.y;
    a.y_ld = g.y_ld;
    a.y_f32 = g.y_f32;
    a.accumulate = g.accumulate;
    a.err = g.err;
    const bool bf16 = g.op == LIN_BF16;
    CUtensorMap mb, ma;
    cudaError_t e;
    if (bf16 && !g.x_mx) {
        e = rows_map(&mb, g.x, g.T, g.K, g.x_ld * 2, a.tile_tokens);
    } else {
        uint16_t *rows = reinterpret_cast<uint16_t *>(g.workspace);
        float *scale = reinterpret_cast<float *>(g.workspace + align256((size_t)g.T * g.K * 2));
        linear_rows_kernel<<<g.T, 256, 0, st>>>(g.x, g.xscales, g.x_ld, g.x_mx, g.K, bf16, rows, scale);
        if ((e = cudaGetLastError()) != cudaSuccess)
            return e;
        a.xscale = scale;
        e = rows_map(&mb, rows, g.T, g.K, (long long)g.K * 2, a.tile_tokens);
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
