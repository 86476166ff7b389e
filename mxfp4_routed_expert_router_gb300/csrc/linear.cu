// linear.cu -- linear layers y = x W^T with MXFP4, group-32 INT4 or BF16
// weights for few tokens (moe_linear_*, include/moe.h): the weight stream is
// read once from the FRAG store and multiplied on the warp-level MMAs.
//
// y[t][n] = sum_k x[t][k] w[n][k].  D[16 weight rows, 8 columns] += A[16, 16] .
// B[16, 8] with weights as A (decoded in registers to FP16; BF16 weights as they
// are) and tokens as B.  For one to four tokens the eight columns of B are not
// left empty: column c = token * NB + blk, NB = 8 / TB blocks of 32 values, so
// that NB consecutive blocks of a row accumulate side by side (B is zero outside
// a column's own block) and their scales are applied once for all of them.
//
// One CTA of 16 warps per SM: with 119 registers a thread, three steps of 2 KB per
// warp are in flight (100 KB an SM; two with INT4 and BF16, whose steps take more
// registers): about what the memory's latency asks for at the full rate.  K is split over clusters where the row groups alone leave SMs idle
// (launch_linear); partial sums meet in a fixed order.
// Bound by HBM for large weights, by the start of the stream (launch, x, the first
// steps' latency: about 3 us) for small ones, and by the decode with more tokens.
// Measured, us per call back to back, over weight copies of 420 MB in all so that none
// stays in L2 (share of a plain copy's bandwidth): MXFP4, one token, 36864 x 7168 23.8
// (0.87), 7168 x 18432 15.1 (0.69), 7168 x 7168 7.7 (0.52; two copies, which stay in L2,
// take as long: the start bounds this size, not HBM); eight tokens 31.8, 21.2, 10.8;
// group-32 INT4, one token, 27.9, 16.5, 8.4; BF16, one token, 7168 x 7168 17.3 (0.88),
// 256 x 7168 3.4.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdio.h>

#include <new>

#include "../../include/moe.h"
#include "gemm_common.cuh"
#include "linear_internal.cuh"
#include "overlap.cuh"

using namespace moe;

struct MoeLinear {
    int N = 0, K = 0, fmt = 0;
    WeightStore frag;         // FRAG / FRAG_F16 layout (few tokens)
    WeightStore tile;         // TILE, TILE_F16 or TILE_I4 layout (the tcgen05 GEMM)
    int op = LIN_BF16;        // the GEMM's operands
    bool stream = true;       // few tokens run on the weight stream (no MXFP4 scale outside its range)
    bool gemm = true;         // more run on the GEMM (INT4: every scale exact relative to its row's base)
    int *err_host = nullptr;  // mapped pinned host memory: [0] device error flag, [1] a rejected scale
                              // at load, [2] an MXFP4 row whose exponents span too widely for FP16 operands,
                              // [3] a scale that one of the two kernels does not take (launch_row_base)
    int *err_dev = nullptr;
};

namespace moe {

namespace {

using gemm::smem_addr;

constexpr int WARPS = 16, THREADS = WARPS * 32;
constexpr int UNIT_BYTES = 16 * CHUNK_K / 2;  // 1024: codes of 16 rows of a chunk

struct LinArgs {
    const uint8_t *w;
    int N, K, kchunks;
    const void *x;
    const uint8_t *xscales;
    long long x_ld;
    int x_mx;           // MXFP8 rows (else BF16)
    int T;
    void *y;
    long long y_ld;
    int y_f32, accumulate;
    int steps;          // steps of K (step_chunks)
    int rgroups;        // groups of 16 rows per CTA
    int xs_off, sum_off, red_off, fin_off;  // shared-memory offsets (bytes), see linear_kernel
};

__device__ __forceinline__ uint4 ldg_stream(const uint8_t *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ uint2 ldg_stream8(const uint8_t *p)
{
    uint2 v;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}

// D += A . B, m16n8k16
template <bool BF>
__device__ __forceinline__ void mma(float d[4], const uint32_t a[4], uint32_t b0, uint32_t b1)
{
    if (BF)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// FRAG_F16 word of E2M1 codes -> A fragment, a hardware conversion per byte
__device__ __forceinline__ void decode_e2m1(uint32_t w, uint32_t a[4])
{
    asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
        " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
        " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}"
        : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
        : "r"(w));
}

// FRAG_F16 word of unsigned 4-bit codes -> A fragment without arithmetic: the
// code in an FP16's lowest bits is the subnormal q * 2^-24 (rows g), in the four
// bits above q * 2^-20 (rows g + 8); the scales undo the powers of two, and the
// zero point is taken off through the block's sum of x.
__device__ __forceinline__ void decode_u4(uint32_t w, uint32_t a[4])
{
    const uint32_t h = w >> 8;
    a[0] = w & 0x000F000Fu;
    a[1] = w & 0x00F000F0u;
    a[2] = h & 0x000F000Fu;
    a[3] = h & 0x00F000F0u;
}

// E8M0 bytes 2H, 2H+1 of w as two floats 2^(e - 127) (exact, also for e = 0)
__device__ __forceinline__ float2 e8m0_pair(uint32_t w16)
{
    uint32_t d;
    asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.bf16x2.ue8m0x2 %0, lo;\n}" : "=r"(d) : "r"(w16));
    return make_float2(__uint_as_float(d << 16), __uint_as_float(d & 0xFFFF0000u));
}

__device__ __forceinline__ float2 half_pair(uint32_t w)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// exponent e of the power of two that FP16 x is divided by, from the bits of
// max |x|: max |x| * 2^-e in [2^14, 2^15), or below for rows of tiny values, whose
// e stops at -127
__device__ __forceinline__ int x_exponent(uint32_t max_bits) { return max((int)(max_bits >> 23) - 141, -127); }

// 2^e for -127 <= e <= 127
__device__ __forceinline__ float pow2f(int e) { return __int_as_float(e < -126 ? 0x400000 : (127 + e) << 23); }

// 8 values of token row t from column k (a multiple of 8; zeros from kend, a
// multiple of 32; from L2, not through the read-only path: the kernel before may
// have written them while this one had started) as they lie in memory: BF16, or E4M3 in x, y and the block's
// E8M0 byte in z.
__device__ __forceinline__ uint4 load_x8(const LinArgs &a, long long t, int k, int kend)
{
    uint4 u = make_uint4(0, 0, 0, 0);
    if (k < kend) {
        if (a.x_mx) {
            const uint2 c = __ldcg(reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(a.x) + t * a.x_ld + k));
            u = make_uint4(c.x, c.y, __ldcg(a.xscales + t * (a.K / 32) + k / 32), 0);
        } else {
            u = __ldcg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.x) + t * a.x_ld + k));
        }
    }
    return u;
}

// E4M3 pairs of load_x8 as FP16 pairs (exact); NaN where the scale byte is 255
__device__ __forceinline__ void e4m3_f16(const uint4 &u, uint32_t h[4])
{
    const uint32_t w[2] = {u.x, u.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint16_t c = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[i]) : "h"(c));
        if (u.z == 255u)
            h[i] = 0x7FFF7FFFu;
    }
}

// The same values as BF16 pairs (E4M3 times a power of two: exact inside BF16's range).
__device__ __forceinline__ void x8_bf16(const LinArgs &a, const uint4 &u, uint32_t o[4])
{
    if (a.x_mx) {
        uint32_t h[4];
        e4m3_f16(u, h);
        const float s = pow2f((int)u.z - 127);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = half_pair(h[i]);
            const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * s, f.y * s);
            o[i] = *reinterpret_cast<const uint32_t *>(&b);
        }
    } else {
        o[0] = u.x, o[1] = u.y, o[2] = u.z, o[3] = u.w;
    }
}

// The same values of a warp's 32 vectors as FP16 pairs times 2^-e, with e from
// the largest of them; returns e.
__device__ __forceinline__ int x8_f16(const LinArgs &a, const uint4 &u, uint32_t o[4])
{
    float f[8];
    float m;
    int es = 0;
    if (a.x_mx) {
        uint32_t h[4];
        e4m3_f16(u, h);
        es = (int)u.z - 127;
        m = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 p = half_pair(h[i]);
            f[2 * i] = p.x;
            f[2 * i + 1] = p.y;
            m = fmaxf(m, fmaxf(fabsf(p.x), fabsf(p.y)));  // (NaN is left out and stays NaN in FP16)
        }
        m *= pow2f(es);
    } else {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        uint32_t mx = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            mx = __vmaxu2(mx, w[i] & 0x7FFF7FFFu);
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
        m = __uint_as_float(max(mx & 0xFFFF0000u, mx << 16));
    }
    const int e = x_exponent(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
    const float mul = pow2f(max(-127, min(127, es - e)));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 hh = __floats2half2_rn(f[2 * i] * mul, f[2 * i + 1] * mul);
        o[i] = *reinterpret_cast<const uint32_t *>(&hh);
    }
    return e;
}

// 16 bytes of shared memory into registers where on != 0 (others keep theirs)
__device__ __forceinline__ void lds16_if(uint32_t on, uint32_t addr, uint32_t r[4])
{
    asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n @p ld.shared.v4.u32 {%0,%1,%2,%3}, [%5];\n}"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3])
                 : "r"(on), "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// chunks of a step of K (256 values with 4-bit weights, 128 with BF16 weights)
template <int FMT>
constexpr int step_chunks = FMT == FMT_BF16 ? 1 : 2;
template <int FMT>
constexpr int chunk_bytes = FMT == FMT_MXFP4 ? CHUNK_MX_BYTES : FMT == FMT_INT4 ? CHUNK_I4_BYTES : CHUNK_BF16_BYTES;

// Registers of one step of 16 rows.  Scales are those of this lane's columns:
// with eight blocks side by side (NB = 8) just the two blocks 2q, 2q + 1 of its
// rows g and g + 8, else every block of both chunks.
template <int FMT, int NB>
struct Step {
    uint4 c[FMT == FMT_BF16 ? 8 : 4];
};
template <int NB>
struct Step<FMT_MXFP4, NB> {
    uint4 c[4];
    uint2 e[2];  // chunk: E8M0 bytes of row g, row g + 8
};
template <>
struct Step<FMT_MXFP4, 8> {
    uint4 c[4];
    uint32_t ea, eb;  // 16 bits each
};
template <int NB>
struct Step<FMT_INT4, NB> {
    uint4 c[4];
    uint4 s[2];  // chunk: FP16 scales of row g (x, y), row g + 8 (z, w)
    uint2 z[2];  // chunk: zero points of row g, row g + 8
};
template <>
struct Step<FMT_INT4, 8> {
    uint4 c[4];
    uint32_t sa, sb, za, zb;
};

// Scales (and zero points) of the lane's columns 2q, 2q + 1 for rows g (a) and
// g + 8 (b) of block group `grp` (NB blocks) of a step.
struct ColScales {
    float2 a, b, za, zb;
};

template <int FMT, int NB>
__device__ __forceinline__ ColScales col_scales(const Step<FMT, NB> &s, int grp, int q)
{
    ColScales r;
    r.za = r.zb = make_float2(0.f, 0.f);
    if constexpr (NB == 8 && FMT == FMT_MXFP4) {
        r.a = e8m0_pair(s.ea);
        r.b = e8m0_pair(s.eb);
    } else if constexpr (NB == 8) {
        r.a = half_pair(s.sa);
        r.b = half_pair(s.sb);
        r.za = make_float2((float)(s.za & 255u), (float)(s.za >> 8));
        r.zb = make_float2((float)(s.zb & 255u), (float)(s.zb >> 8));
    } else {
        const int h = grp * NB / 4;  // chunk
        // which half of the chunk's four blocks: NB = 4 by lane, else by group
        const bool second = NB == 4 ? (q & 1) != 0 : NB == 2 ? (grp & 1) != 0 : ((grp & 3) >> 1) != 0;
        if constexpr (FMT == FMT_MXFP4) {
            r.a = e8m0_pair(second ? s.e[h].x >> 16 : s.e[h].x);
            r.b = e8m0_pair(second ? s.e[h].y >> 16 : s.e[h].y);
        } else {
            r.a = half_pair(second ? s.s[h].y : s.s[h].x);
            r.b = half_pair(second ? s.s[h].w : s.s[h].z);
            const uint32_t z0 = second ? s.z[h].x >> 16 : s.z[h].x, z1 = second ? s.z[h].y >> 16 : s.z[h].y;
            r.za = make_float2((float)(z0 & 255u), (float)((z0 >> 8) & 255u));
            r.zb = make_float2((float)(z1 & 255u), (float)((z1 >> 8) & 255u));
        }
        if constexpr (NB == 1) {  // both columns are the same block
            const bool odd = grp & 1;
            r.a.x = r.a.y = odd ? r.a.y : r.a.x;
            r.b.x = r.b.y = odd ? r.b.y : r.b.x;
            r.za.x = r.za.y = odd ? r.za.y : r.za.x;
            r.zb.x = r.zb.y = odd ? r.zb.y : r.zb.x;
        }
    }
    return r;
}

// Steps are cut evenly: warp w of n takes steps [w * units / n, (w + 1) * units
// / n) of the CTA's row groups laid end to end; the warp that holds step u:
__device__ __forceinline__ int owner_of(int u, int units, int n) { return ((u + 1) * n - 1) / units; }

// One CTA: `rgroups` groups of 16 rows (fewer at the end), its K range (the
// whole of K, or a share of a cluster's), up to TB tokens.  x is staged
// once; then every warp streams its share of the CTA's steps with DEPTH of them
// in flight and writes a partial sum for each row group that it touches.
// blockIdx.x = row tile * cluster size + rank.
template <int FMT, int TB>
__global__ void __launch_bounds__(THREADS, 1) linear_kernel(const __grid_constant__ LinArgs a)
{
    constexpr int NB = 8 / TB;         // blocks side by side in the columns of one n-tile
    constexpr bool BF = FMT == FMT_BF16;
    constexpr int SC = step_chunks<FMT>, SB = SC * 4;  // chunks and 32-value blocks of a step
    constexpr int BLK_BYTES = TB * 64;                 // B fragments of a block
    constexpr int CB = chunk_bytes<FMT>;
    extern __shared__ __align__(16) uint8_t smem[];
    uint8_t *xf = smem;                                              // B fragments
    float *xscale = reinterpret_cast<float *>(smem + a.xs_off);      // [256 values][TB] powers of two
    float *xsum = reinterpret_cast<float *>(smem + a.sum_off);       // INT4: [block][TB] sums of the FP16 values
    float *red = reinterpret_cast<float *>(smem + a.red_off);        // [warp + row group][token][16]
    float *fin = reinterpret_cast<float *>(smem + a.fin_off);        // [row group][token][16] (clusters)
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
    overlap_trigger();
    uint32_t crank, csize;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(crank));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(csize));
    const int n16 = (a.N + 15) / 16;
    const int rg0 = (int)(blockIdx.x / csize) * a.rgroups;
    const int R = min(a.rgroups, n16 - rg0);
    const int p0 = (int)((long long)a.steps * crank / csize), p1 = (int)((long long)a.steps * (crank + 1) / csize);
    const int P = p1 - p0;
    const int tv = a.T;  // at most TB
    const int units = R * P, nw = min(WARPS, units);
    const int u0 = nw ? min(units, warp * units / nw) : 0, u1 = nw ? min(units, (warp + 1) * units / nw) : 0;

    // ---- weights of this warp's first steps are in flight while x is staged.
    // A step past the row's last chunk (an odd number of chunks) reads what
    // follows in the store: x is zero there, and every code and scale is finite.
    int lu = u0, lr = P ? u0 / P : 0, lp = P ? u0 % P : 0;  // load cursor: step, its row group and place in K
    const uint8_t *wp = nullptr;  // the cursor's chunk
    int w8 = 0;
    auto locate = [&]() {
        const int rg = rg0 + lr;
        w8 = rg & 7;
        wp = a.w + ((size_t)(rg >> 3) * a.kchunks + (size_t)(p0 + lp) * SC) * CB;
    };
    if (u0 < u1)
        locate();
    auto load = [&](Step<FMT, NB> &s) {
        if (lu >= u1)
            return;
        const uint8_t *code = wp + w8 * (BF ? 4096 : UNIT_BYTES) + lane * 16;
        if constexpr (BF) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                s.c[j] = ldg_stream(code + j * 512);
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                s.c[2 * h] = ldg_stream(code + h * CB);
                s.c[2 * h + 1] = ldg_stream(code + h * CB + 512);
            }
            const uint8_t *sc = wp + CHUNK_MX_CODE_BYTES;
            const int row = w8 * 8 + g;
            if constexpr (FMT == FMT_MXFP4 && NB == 8) {
                const uint8_t *p = sc + (q >> 1) * CB + row * 8 + (q & 1) * 2;
                s.ea = __ldg(reinterpret_cast<const uint16_t *>(p));
                s.eb = __ldg(reinterpret_cast<const uint16_t *>(p + 4));
            } else if constexpr (FMT == FMT_MXFP4) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    s.e[h] = ldg_stream8(sc + h * CB + row * 8);
            } else if constexpr (NB == 8) {
                const uint8_t *p = sc + (q >> 1) * CB + row * 16 + (q & 1) * 4;
                s.sa = __ldg(reinterpret_cast<const uint32_t *>(p));
                s.sb = __ldg(reinterpret_cast<const uint32_t *>(p + 8));
                const uint8_t *z = sc + (q >> 1) * CB + CHUNK_I4_SCALE_BYTES + row * 8 + (q & 1) * 2;
                s.za = __ldg(reinterpret_cast<const uint16_t *>(z));
                s.zb = __ldg(reinterpret_cast<const uint16_t *>(z + 4));
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    s.s[h] = ldg_stream(sc + h * CB + row * 16);
                    s.z[h] = ldg_stream8(sc + h * CB + CHUNK_I4_SCALE_BYTES + row * 8);
                }
            }
        }
        ++lu;
        wp += SC * CB;
        if (++lp == P) {
            lp = 0;
            ++lr;
            locate();
        }
    };
    // ---- x: this CTA's columns of the tile's tokens as B fragments [block][token]
    // [64 bytes].  An item is 256 values of one token, a vector of 8 per lane; a
    // warp loads XB items at a time.  FP16 operands
    // take x * 2^-e, e from the item's largest |x| (in [2^14, 2^15) then): exact for
    // BF16 and E4M3 values within 2^-29 of it.
    constexpr int XB = 4;
    const int items = (P * SB + 7) / 8 * TB;
    const int k0 = p0 * SC * CHUNK_K;
    const int kend = min(a.K, k0 + P * SC * CHUNK_K);
    uint4 xr[XB];
    auto load_items = [&](int i0) {
#pragma unroll
        for (int b = 0; b < XB; ++b) {
            const int i = i0 + b * WARPS, t = i % TB;
            if (i < items && t < tv)
                xr[b] = load_x8(a, t, k0 + (i / TB * 32 + lane) * 8, kend);
        }
    };
    constexpr int DEPTH = FMT == FMT_MXFP4 ? 3 : 2;  // (three spill with INT4: 33 against 27 us at 7168 x 18432, 8 tokens)
    Step<FMT, NB> st[DEPTH];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
        load(st[d]);
    overlap_wait();
    load_items(warp);
    for (int i0 = warp; i0 < items; i0 += XB * WARPS) {
#pragma unroll
        for (int b = 0; b < XB; ++b) {
            const int i = i0 + b * WARPS, t = i % TB;
            if (i >= items || t >= tv)
                continue;
            const int c = i / TB * 32 + lane;  // vector of 8 values in this CTA's columns
            uint32_t o[4];
            if (BF) {
                x8_bf16(a, xr[b], o);
            } else {
                const int e = x8_f16(a, xr[b], o);
                if (lane == 0)
                    xscale[i] = pow2f(e);
                if (FMT == FMT_INT4) {
                    float s = 0.f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 f = half_pair(o[j]);
                        s += f.x + f.y;
                    }
                    // four vectors (adjacent lanes) make a block
                    s += __shfl_xor_sync(0xffffffffu, s, 1);
                    s += __shfl_xor_sync(0xffffffffu, s, 2);
                    if ((lane & 3) == 0)
                        xsum[(c >> 2) * TB + t] = s;
                }
            }
            // values 8c .. 8c+7 of the row: k step (c & 3) / 2 of the block, low or high eight
            uint8_t *dst = xf + ((c >> 2) * TB + t) * 64 + ((c >> 1) & 1) * 8 + (c & 1) * 4;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<uint32_t *>(dst + j * 16) = o[j];
        }
        load_items(i0 + XB * WARPS);
    }
    __syncthreads();

    // ---- weight stream
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    // B column g of the lane: token g / NB, block g % NB of a group; NB > 1: B of
    // block i is zero in the lanes of the other columns, which never load it
    uint32_t bx[NB][4];
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            bx[i][j] = 0u;
    const uint32_t xb0 = smem_addr(xf) + (g / NB) * 64 + q * 16;
    auto compute = [&](const Step<FMT, NB> &s, int p) {
        const uint32_t *cw = reinterpret_cast<const uint32_t *>(s.c);
        const uint32_t xb = xb0 + p * (SB * BLK_BYTES);
        float sum[4];  // of the step, in units of the tokens' powers of two
#pragma unroll
        for (int grp = 0; grp < SB / NB; ++grp) {
            float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int blk = grp * NB + i;
                uint32_t a0[4], a1[4];
                if constexpr (BF) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        a0[j] = cw[8 * blk + j];
                        a1[j] = cw[8 * blk + 4 + j];
                    }
                } else if constexpr (FMT == FMT_MXFP4) {
                    decode_e2m1(cw[2 * blk], a0);
                    decode_e2m1(cw[2 * blk + 1], a1);
                } else {
                    decode_u4(cw[2 * blk], a0);
                    decode_u4(cw[2 * blk + 1], a1);
                }
                uint32_t *b = bx[i];
                lds16_if(NB == 1 || g % NB == i, xb + blk * BLK_BYTES, b);
                mma<BF>(BF ? acc : part, a0, b[0], b[1]);
                mma<BF>(BF ? acc : part, a1, b[2], b[3]);
            }
            if constexpr (!BF) {
                const ColScales cs = col_scales<FMT, NB>(s, grp, q);
                if (FMT == FMT_INT4) {
                    // sum q x - z sum x, then the group's scale
                    const int c0 = 2 * q, c1 = 2 * q + 1;
                    const float *xs = xsum + (p * SB + grp * NB) * TB;
                    const float x0 = xs[(c0 % NB) * TB + c0 / NB], x1 = xs[(c1 % NB) * TB + c1 / NB];
                    part[0] = fmaf(part[0], 16777216.f, -cs.za.x * x0);
                    part[1] = fmaf(part[1], 16777216.f, -cs.za.y * x1);
                    part[2] = fmaf(part[2], 1048576.f, -cs.zb.x * x0);
                    part[3] = fmaf(part[3], 1048576.f, -cs.zb.y * x1);
                }
                sum[0] = grp ? fmaf(part[0], cs.a.x, sum[0]) : part[0] * cs.a.x;
                sum[1] = grp ? fmaf(part[1], cs.a.y, sum[1]) : part[1] * cs.a.y;
                sum[2] = grp ? fmaf(part[2], cs.b.x, sum[2]) : part[2] * cs.b.x;
                sum[3] = grp ? fmaf(part[3], cs.b.y, sum[3]) : part[3] * cs.b.y;
            }
        }
        if constexpr (!BF) {
            const float *xs = xscale + p * TB;
            const float x0 = xs[2 * q / NB], x1 = xs[(2 * q + 1) / NB];
            acc[0] = fmaf(sum[0], x0, acc[0]);
            acc[1] = fmaf(sum[1], x1, acc[1]);
            acc[2] = fmaf(sum[2], x0, acc[2]);
            acc[3] = fmaf(sum[3], x1, acc[3]);
        }
    };
    // partial sums of row group r (of the CTA): summed over the blocks side by side
    auto flush = [&](int r) {
        float *o = red + (size_t)(warp + r) * TB * 16;
        if (NB == 1) {
            o[(2 * q) * 16 + g] = acc[0];
            o[(2 * q + 1) * 16 + g] = acc[1];
            o[(2 * q) * 16 + g + 8] = acc[2];
            o[(2 * q + 1) * 16 + g + 8] = acc[3];
        } else {
            float r0 = acc[0] + acc[1], r1 = acc[2] + acc[3];
            if (NB >= 4) {
                r0 += __shfl_xor_sync(0xffffffffu, r0, 1);
                r1 += __shfl_xor_sync(0xffffffffu, r1, 1);
            }
            if (NB == 8) {
                r0 += __shfl_xor_sync(0xffffffffu, r0, 2);
                r1 += __shfl_xor_sync(0xffffffffu, r1, 2);
            }
            const int tok = 2 * q / NB;
            if (2 * q % NB == 0) {  // one of the lanes that share a token
                o[tok * 16 + g] = r0;
                o[tok * 16 + g + 8] = r1;
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[j] = 0.f;
    };
    int r = P ? u0 / P : 0, p = P ? u0 % P : 0;
    for (int u = u0; u < u1; u += DEPTH) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            if (u + d < u1) {
                compute(st[d], p);
                load(st[d]);
                if (++p == P || u + d + 1 == u1) {
                    flush(r);
                    p = 0;
                    ++r;
                }
            }
        }
    }
    __syncthreads();

    // ---- sums over the warps that share a row group, then over the cluster, in
    // a fixed order
    const int total = R * tv * 16;
    auto store = [&](int i, float v) {
        const int rt = i >> 4, rr = rt / tv;
        const int n = (rg0 + rr) * 16 + (i & 15);
        if (n < a.N) {
            const long long at = (long long)(rt - rr * tv) * a.y_ld + n;
            if (a.y_f32) {
                float *y = static_cast<float *>(a.y) + at;
                *y = a.accumulate ? *y + v : v;
            } else {
                static_cast<__nv_bfloat16 *>(a.y)[at] = __float2bfloat16_rn(v);
            }
        }
    };
    for (int i = tid; i < total; i += THREADS) {
        const int rt = i >> 4, rr = rt / tv, t = rt - rr * tv;
        float v = 0.f;
        if (P) {
            const int w1 = owner_of((rr + 1) * P - 1, units, nw);
            for (int w = owner_of(rr * P, units, nw); w <= w1; ++w)
                v += red[(size_t)((w + rr) * TB + t) * 16 + (i & 15)];
        }
        if (csize == 1)
            store(i, v);
        else
            fin[i] = v;
    }
    if (csize == 1)
        return;
    cluster_sync();
    // rank r finishes every csize-th run of THREADS sums
    for (int i = crank * THREADS + tid; i < total; i += csize * THREADS) {
        float v = 0.f;
        const uint32_t local = (uint32_t)__cvta_generic_to_shared(fin + i);
        for (uint32_t rk = 0; rk < csize; ++rk) {
            uint32_t remote;
            float f;
            asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rk));
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f) : "r"(remote));
            v += f;
        }
        store(i, v);
    }
    cluster_sync();  // a CTA's sums stay in place until every rank has read them
}

// ------------------------------------------------------------------ host side

// How a call is cut: a cluster of `cluster` CTAs along K, `rgroups` groups of 16
// rows per cluster, and a CTA's shared memory.
struct Cut {
    int cluster, rgroups, smem, xs_off, sum_off, red_off, fin_off;
};

constexpr int SMEM_MAX = 220 * 1024;

Cut cut_of(int n16, int steps, int step_blocks, int tt, int tv, bool i4, int cluster, int slots)
{
    Cut c;
    c.cluster = cluster;
    const int segs = ((steps + cluster - 1) / cluster * step_blocks + 7) / 8;  // x is staged by 256 values
    c.xs_off = segs * 8 * tt * 64;
    c.sum_off = c.xs_off + segs * tt * 4;
    c.red_off = (c.sum_off + (i4 ? segs * 8 * tt * 4 : 0) + 15) & ~15;
    // one wave of clusters where the partial sums of its row groups fit
    const int per = tt * 16 * 4, room = SMEM_MAX - c.red_off - WARPS * per;
    c.rgroups = (n16 + slots - 1) / slots;
    const int most = room > 0 ? room / (per + (cluster > 1 ? tv * 64 : 0)) : 0;
    if (c.rgroups > most)
        c.rgroups = most;
    c.fin_off = c.red_off + (WARPS + c.rgroups) * per;
    c.smem = c.fin_off + (cluster > 1 ? c.rgroups * tv * 64 : 0);
    return c;
}

// Clusters of `size` CTAs of a kernel that the current device runs at a time (one
// CTA per SM: the register file holds one), looked up once per device.
template <int FMT, int TB>
int clusters_of(int size)
{
    const int sms = gemm::sm_count();
    if (size == 1)
        return sms;
    static std::atomic<int> cached[gemm::MAX_DEVICES][4];
    const int dev = gemm::current_device(), at = size == 2 ? 1 : size == 4 ? 2 : 3;
    const bool cacheable = dev >= 0 && dev < gemm::MAX_DEVICES;
    int n = cacheable ? cached[dev][at].load(std::memory_order_relaxed) : 0;
    if (n > 0)
        return n;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(sms / size * size);
    cfg.blockDim = dim3(THREADS);
    cudaLaunchAttribute at_cl;
    at_cl.id = cudaLaunchAttributeClusterDimension;
    at_cl.val.clusterDim.x = (unsigned)size;
    at_cl.val.clusterDim.y = at_cl.val.clusterDim.z = 1;
    cfg.attrs = &at_cl;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, linear_kernel<FMT, TB>, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();
        n = sms / size > 0 ? sms / size : 1;
    }
    if (cacheable)
        cached[dev][at].store(n, std::memory_order_relaxed);
    return n;
}

template <int FMT, int TB>
cudaError_t launch_linear(const LinArgs &args, cudaStream_t st)
{
    constexpr int SC = step_chunks<FMT>;
    LinArgs a = args;
    a.steps = (a.kchunks + SC - 1) / SC;
    const int n16 = (a.N + 15) / 16;
    // The cluster size with the least estimated time, of those whose shared memory
    // holds x: a CTA's steps (0.05 us each, more with several tokens), its items of x
    // (1/16 of a warp's 0.25 us) and the cluster's barriers.
    Cut best{};
    double least = 0.;
    for (int cl = 1; cl <= 8 && (cl == 1 || cl <= a.steps); cl *= 2) {
        const int slots = clusters_of<FMT, TB>(cl);
        const Cut c = cut_of(n16, a.steps, SC * 4, TB, a.T, FMT == FMT_INT4, cl, slots);
        if (c.rgroups < 1)
            continue;
        const int grid = (n16 + c.rgroups - 1) / c.rgroups;
        const int waves = (grid + slots - 1) / slots;
        const double steps = (double)((a.steps + cl - 1) / cl);
        const double us = waves * (c.rgroups * steps * (0.05 + 0.003 * TB) + steps * SC * TB / 2 * 0.016 +
                                   (cl > 1 ? 1.0 + 0.1 * cl : 0.));
        if (best.rgroups < 1 || us < least) {
            least = us;
            best = c;
        }
    }
    if (best.rgroups < 1)
        return cudaErrorInvalidValue;
    a.rgroups = best.rgroups;
    a.xs_off = best.xs_off;
    a.sum_off = best.sum_off;
    a.red_off = best.red_off;
    a.fin_off = best.fin_off;
    auto kern = linear_kernel<FMT, TB>;
    static std::atomic<int> attr_set[gemm::MAX_DEVICES];
    cudaError_t e = gemm::smem_limit_once(attr_set, (const void *)kern, SMEM_MAX);
    if (e != cudaSuccess)
        return e;
    return launch_overlapped(kern, (unsigned)((n16 + best.rgroups - 1) / best.rgroups * best.cluster), THREADS, best.smem,
                             best.cluster, st, a);
}

template <int FMT>
cudaError_t launch_tokens(const LinArgs &a, cudaStream_t st)
{
    if constexpr (FMT != FMT_BF16) {  // (BF16 weights have no scales to apply per block)
        if (a.T == 1)
            return launch_linear<FMT, 1>(a, st);
        if (a.T == 2)
            return launch_linear<FMT, 2>(a, st);
        if (a.T <= 4)
            return launch_linear<FMT, 4>(a, st);
    }
    return launch_linear<FMT, 8>(a, st);
}

MoeStatus bad(MoeStatus s, const char *msg) { return (MoeStatus)set_last_error(s, msg); }

MoeStatus bad_cuda(const char *what, cudaError_t e)
{
    char msg[160];
    snprintf(msg, sizeof msg, "%s: %s", what, cudaGetErrorString(e));
    return bad(MOE_ECUDA, msg);
}

// Whether T tokens run on the weight stream: few of them, or, without the GEMM, any number in slices of few.
bool on_stream(const MoeLinear *l, int T) { return (T <= LINEAR_STREAM_MAX_T && l->stream) || !l->gemm; }

void destroy(MoeLinear *l)
{
    if (l->frag.base)
        cudaFree(l->frag.base);
    if (l->tile.base)
        cudaFree(l->tile.base);
    if (l->tile.row_base)
        cudaFree(l->tile.row_base);
    if (l->err_host)
        cudaFreeHost(l->err_host);
    delete l;
}

}  // namespace

}  // namespace moe

extern "C" {

MoeStatus moe_linear_load(int N, int K, MoeWeightFormat wfmt, const MoeMx *w, void *cuda_stream, MoeLinear **out)
{
    char msg[160];
    if (!w || !out)
        return bad(MOE_EINVAL, "moe_linear_load: NULL argument");
    if (wfmt != MOE_W_MXFP4 && wfmt != MOE_W_BF16 && wfmt != MOE_W_INT4G32) {
        snprintf(msg, sizeof msg, "unknown weight format %d", (int)wfmt);
        return bad(MOE_EINVAL, msg);
    }
    if (N < 1 || N > (1 << 20)) {
        snprintf(msg, sizeof msg, "N = %d out of range [1, 2^20]", N);
        return bad(MOE_EINVAL, msg);
    }
    if (K < 32 || K % 32 || K > 65536) {
        snprintf(msg, sizeof msg, "K (%d) must be a multiple of 32 in 32 .. 65536", K);
        return bad(MOE_EDIMS, msg);
    }
    const int fmt = wfmt == MOE_W_MXFP4 ? FMT_MXFP4 : wfmt == MOE_W_INT4G32 ? FMT_INT4 : FMT_BF16;
    if (!w->codes || (fmt != FMT_BF16 && !w->scales))
        return bad(MOE_EINVAL, "moe_linear_load: the weight has a NULL pointer");
    if (fmt == FMT_INT4 && (uintptr_t)w->scales % 2)
        return bad(MOE_EINVAL, "moe_linear_load: scales (FP16) are not 2-byte aligned");
    MoeLinear *l = new (std::nothrow) MoeLinear();
    if (!l)
        return bad(MOE_ENOMEM, "host allocation failed");
    l->N = N;
    l->K = K;
    l->fmt = fmt;
    cudaStream_t st = (cudaStream_t)cuda_stream;
    WeightStore &f = l->frag;
    f.rows = N;
    f.cols = K;
    f.row_tiles = (N + TILE_ROWS - 1) / TILE_ROWS;
    f.kchunks = (K + CHUNK_K - 1) / CHUNK_K;
    f.chunk_bytes = fmt == FMT_MXFP4 ? CHUNK_MX_BYTES : fmt == FMT_INT4 ? CHUNK_I4_BYTES : CHUNK_BF16_BYTES;
    f.group_bytes = (size_t)f.row_tiles * f.kchunks * f.chunk_bytes;
    cudaError_t e;
    if ((e = cudaHostAlloc((void **)&l->err_host, 4 * sizeof(int), cudaHostAllocMapped)) != cudaSuccess) {
        destroy(l);
        return bad_cuda("cudaHostAlloc", e);
    }
    for (int i = 0; i < 4; ++i)
        l->err_host[i] = 0;
    if ((e = cudaHostGetDevicePointer((void **)&l->err_dev, l->err_host, 0)) != cudaSuccess) {
        destroy(l);
        return bad_cuda("cudaHostGetDevicePointer", e);
    }
    WeightStore &t = l->tile;
    t = f;
    // two copies, one for each kernel; a step of two chunks may read one past a row
    // tile's last (see linear_kernel)
    const size_t bytes = f.group_bytes + f.chunk_bytes;
    if (cudaMalloc(&f.base, bytes) != cudaSuccess || cudaMalloc(&t.base, t.group_bytes) != cudaSuccess ||
        (fmt != FMT_BF16 && cudaMalloc(&t.row_base, (size_t)t.row_tiles * TILE_ROWS) != cudaSuccess)) {
        cudaGetLastError();
        snprintf(msg, sizeof msg, "device allocation of %zu bytes of weights failed", bytes + t.group_bytes);
        destroy(l);
        return bad(MOE_ENOMEM, msg);
    }
    const SrcMat src = {(const uint8_t *)w->codes, (const uint8_t *)(fmt == FMT_BF16 ? nullptr : w->scales),
                        fmt == FMT_BF16 ? (long long)K * 2 : K / 2, K / 32,
                        (const uint8_t *)(fmt == FMT_INT4 ? w->zeros : nullptr)};
    if ((fmt != FMT_BF16 &&
         (e = launch_row_base(fmt, false, src, src, t, 0, K, N, &l->err_dev[2], st, &l->err_dev[3])) != cudaSuccess) ||
        (e = cudaMemsetAsync(f.base + f.group_bytes, 0, f.chunk_bytes, st)) != cudaSuccess ||
        (e = launch_repack(fmt, fmt == FMT_BF16 ? LAYOUT_FRAG : LAYOUT_FRAG_F16, false, src, src, f, 0, K, N,
                           &l->err_dev[1], st)) != cudaSuccess ||
        (e = cudaStreamSynchronize(st)) != cudaSuccess) {
        destroy(l);
        return bad_cuda("repack", e);
    }
    if (*(volatile int *)&l->err_host[3])
        (fmt == FMT_INT4 ? l->gemm : l->stream) = false;
    int layout = LAYOUT_TILE;
    if (fmt == FMT_INT4) {
        l->op = LIN_I4;
        layout = LAYOUT_TILE_I4;
    } else if (fmt == FMT_MXFP4 && *(volatile int *)&l->err_host[2] == 0) {
        l->op = LIN_F16;
        layout = LAYOUT_TILE_F16;
    }
    if ((e = launch_repack(fmt, layout, false, src, src, t, 0, K, N, &l->err_dev[1], st)) != cudaSuccess ||
        (e = cudaStreamSynchronize(st)) != cudaSuccess) {
        destroy(l);
        return bad_cuda("repack", e);
    }
    if (*(volatile int *)&l->err_host[1]) {
        destroy(l);
        return bad(MOE_ESCALE, fmt == FMT_INT4 ? "an INT4 FP16 scale is Inf or NaN, or a zero point is above 15"
                                               : "an E8M0 scale byte is 255 (NaN)");
    }
    *out = l;
    return MOE_OK;
}

size_t moe_linear_workspace_bytes(const MoeLinear *l, int T)
{
    return !l || T <= 0 || on_stream(l, T) ? 0 : linear_gemm_workspace(l->K, T);
}

MoeStatus moe_linear_forward(MoeLinear *l, const void *x, MoeRowType x_type, long long x_ld, const void *x_scales,
                             int T, void *y, MoeRowType y_type, long long y_ld, int accumulate, void *workspace,
                             size_t ws_bytes, void *cuda_stream)
{
    char msg[160];
    if (!l)
        return bad(MOE_EINVAL, "moe_linear_forward: NULL handle");
    if (T < 0 || T > (1 << 20)) {
        snprintf(msg, sizeof msg, "T = %d out of range [0, 2^20]", T);
        return bad(MOE_EINVAL, msg);
    }
    if (x_type != MOE_ROWS_BF16 && x_type != MOE_ROWS_MXFP8)
        return bad(MOE_EINVAL, "moe_linear_forward: x is BF16 or MXFP8");
    if (y_type != MOE_ROWS_BF16 && y_type != MOE_ROWS_F32)
        return bad(MOE_EINVAL, "moe_linear_forward: y is F32 or BF16");
    if (accumulate && y_type != MOE_ROWS_F32)
        return bad(MOE_EINVAL, "moe_linear_forward: only F32 rows accumulate");
    const int err = *(volatile int *)l->err_host;
    if (err != DEV_ERR_NONE) {
        snprintf(msg, sizeof msg, "a kernel of an earlier call reported device error %d", err);
        return bad(MOE_EDEVICE, msg);
    }
    if (T == 0)
        return MOE_OK;
    if (!x || !y || (x_type == MOE_ROWS_MXFP8 && !x_scales))
        return bad(MOE_EINVAL, "moe_linear_forward: NULL pointer");
    if (x_ld < l->K || y_ld < l->N)
        return bad(MOE_EINVAL, "moe_linear_forward: a row stride is below the row's length");
    if ((uintptr_t)x % 16 || x_ld * (x_type == MOE_ROWS_BF16 ? 2 : 1) % 16)
        return bad(MOE_EINVAL, "moe_linear_forward: rows of x must start on 16-byte boundaries");
    if ((uintptr_t)y % (y_type == MOE_ROWS_F32 ? 4 : 2))
        return bad(MOE_EINVAL, "moe_linear_forward: y is misaligned");
    // (the GEMM reads the caller's BF16 rows as they are with BF16 weights, else rows that it writes first)
    const bool rows = l->fmt != FMT_BF16 || x_type == MOE_ROWS_MXFP8;
    if (rows && ws_bytes < moe_linear_workspace_bytes(l, T))
        return bad(MOE_EWORKSPACE, "moe_linear_forward: the workspace is smaller than moe_linear_workspace_bytes");
    if ((uintptr_t)workspace % 256)
        return bad(MOE_EWORKSPACE, "moe_linear_forward: the workspace must be 256-byte aligned");
    cudaStream_t st = (cudaStream_t)cuda_stream;
    if (!on_stream(l, T)) {
        if (rows && !workspace)
            return bad(MOE_EWORKSPACE, "moe_linear_forward: NULL workspace");
        LinearGemm g{};
        g.w = &l->tile;
        g.fmt = l->fmt;
        g.op = l->op;
        g.N = l->N;
        g.K = l->K;
        g.T = T;
        g.x = x;
        g.xscales = (const uint8_t *)x_scales;
        g.x_ld = x_ld;
        g.x_mx = x_type == MOE_ROWS_MXFP8;
        g.y = y;
        g.y_ld = y_ld;
        g.y_f32 = y_type == MOE_ROWS_F32;
        g.accumulate = accumulate != 0;
        g.workspace = (uint8_t *)workspace;
        g.err = l->err_dev;
        const cudaError_t e = launch_linear_gemm(g, st);
        return e == cudaSuccess ? MOE_OK : bad_cuda("linear layer launch", e);
    }
    LinArgs a{};
    a.w = l->frag.base;
    a.N = l->N;
    a.K = l->K;
    a.kchunks = l->frag.kchunks;
    a.x_ld = x_ld;
    a.x_mx = x_type == MOE_ROWS_MXFP8;
    a.y_ld = y_ld;
    a.y_f32 = y_type == MOE_ROWS_F32;
    a.accumulate = accumulate != 0;
    for (int t = 0; t < T; t += LINEAR_STREAM_MAX_T) {  // (once, but for INT4 weights that the GEMM does not take)
        a.T = T - t < LINEAR_STREAM_MAX_T ? T - t : LINEAR_STREAM_MAX_T;
        a.x = (const uint8_t *)x + t * x_ld * (a.x_mx ? 1 : 2);
        a.xscales = a.x_mx ? (const uint8_t *)x_scales + (long long)t * (l->K / 32) : nullptr;
        a.y = (uint8_t *)y + t * y_ld * (a.y_f32 ? 4 : 2);
        const cudaError_t e = l->fmt == FMT_MXFP4  ? launch_tokens<FMT_MXFP4>(a, st)
                              : l->fmt == FMT_INT4 ? launch_tokens<FMT_INT4>(a, st)
                                                   : launch_tokens<FMT_BF16>(a, st);
        if (e != cudaSuccess)
            return bad_cuda("linear layer launch", e);
    }
    return MOE_OK;
}

MoeStatus moe_linear_sync_status(MoeLinear *l, void *cuda_stream)
{
    if (!l)
        return bad(MOE_EINVAL, "moe_linear_sync_status: NULL handle");
    const cudaError_t e = cudaStreamSynchronize((cudaStream_t)cuda_stream);
    if (e != cudaSuccess)
        return bad_cuda("cudaStreamSynchronize", e);
    const int err = *(volatile int *)l->err_host;
    if (err != DEV_ERR_NONE) {
        char msg[96];
        snprintf(msg, sizeof msg, "a kernel reported device error %d", err);
        return bad(MOE_EDEVICE, msg);
    }
    return MOE_OK;
}

void moe_linear_free(MoeLinear *l)
{
    if (!l)
        return;
    cudaDeviceSynchronize();
    destroy(l);
}

}  // extern "C"
