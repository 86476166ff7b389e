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
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdio.h>

#include <new>

#include "../../include/moe.h"
#include "gemm_common.cuh"
#include "moe_internal.cuh"

using namespace moe;

struct MoeLinear {
    int N = 0, K = 0, fmt = 0;
    WeightStore frag;         // FRAG / FRAG_F16 layout
    int *err_host = nullptr;  // mapped pinned host memory: [0] device error flag, [1] a rejected scale at load
    int *err_dev = nullptr;
};

namespace moe {

namespace {

constexpr int WARPS = 8, THREADS = WARPS * 32;
constexpr int UNIT_BYTES = 16 * CHUNK_K / 2;  // 1024: codes of 16 rows of a chunk

struct LinArgs {
    const uint8_t *w;
    int N, K, kchunks, chunk_bytes;
    const void *x;
    const uint8_t *xscales;
    long long x_ld;
    int x_mx;           // MXFP8 rows (else BF16)
    int T;
    void *y;
    long long y_ld;
    int y_f32, accumulate;
    int kw;             // warps of a CTA that split its K range (1, 2, 4, 8)
    int pairs;          // 256-value steps of K: ceil(kchunks / 2)
    int xs_off, red_off;  // shared-memory offsets (bytes) of the token scales and block sums, and of the partial sums
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

// 2^e as a product of two floats for any e that the callers have (|e| <= 252)
__device__ __forceinline__ float scale_pow2(float v, int e)
{
    const int h = e / 2;
    return v * __int_as_float((127 + h) << 23) * __int_as_float((127 + e - h) << 23);
}

// 8 values of token row t from column k (k and K are multiples of 8 and 32; zeros past K)
__device__ __forceinline__ void load_x8(const LinArgs &a, long long t, int k, float v[8])
{
    if (k >= a.K) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = 0.f;
        return;
    }
    if (a.x_mx) {
        const uint2 u = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(a.x) + t * a.x_ld + k));
        const int e = __ldg(a.xscales + t * (a.K / 32) + k / 32);
        const float s = e == 255 ? __int_as_float(0x7FC00000) : __int_as_float(e ? e << 23 : 0x400000);
        const uint32_t w[2] = {u.x, u.y};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint16_t c = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
            uint32_t h;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
            const float2 f = half_pair(h);
            v[2 * i] = f.x * s;
            v[2 * i + 1] = f.y * s;
        }
    } else {
        const uint4 u =
            __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.x) + t * a.x_ld + k));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// registers of one 256-value step of 16 rows
template <int FMT>
struct Step {
    uint4 c[FMT == FMT_BF16 ? 16 : 4];
    uint4 s[2];  // INT4: FP16 scales of both chunks; MXFP4: E8M0 bytes in .x, .y
    uint2 z[2];  // INT4: zero points
};

// One CTA: WARPS / kw groups of 16 rows, its K range (the whole of K, or a
// share of a cluster's) split over kw warps by steps of 256 values; up to TB * NT
// tokens.  blockIdx.x = row tile * cluster size + rank, blockIdx.y = token tile.
template <int FMT, int TB, int NT>
__global__ void __launch_bounds__(THREADS) linear_kernel(const LinArgs a)
{
    constexpr int NB = 8 / TB;         // blocks side by side in the columns of one n-tile
    constexpr bool BF = FMT == FMT_BF16;
    constexpr int TT = TB * NT;        // tokens of a tile
    static_assert(NT == 1 || TB == 8, "several n-tiles hold 8 tokens each");
    extern __shared__ __align__(16) uint8_t smem[];
    uint8_t *xf = smem;                                              // B fragments: [block][token][64 bytes]
    int *xmax = reinterpret_cast<int *>(smem + a.xs_off);            // [TT] bits of max |x|
    float *xsum = reinterpret_cast<float *>(smem + a.xs_off + 64);   // INT4: [block][token] sums of the FP16 values
    float *red = reinterpret_cast<float *>(smem + a.red_off);        // [kw][token][rows of the CTA]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
    uint32_t crank, csize;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(crank));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(csize));
    const int rgroups = WARPS / a.kw;
    const int tile = blockIdx.x / csize;
    const int kwi = warp % a.kw, rwi = warp / a.kw;
    const int rg = tile * rgroups + rwi;  // this warp's group of 16 rows
    const int p0 = (int)((long long)a.pairs * crank / csize), p1 = (int)((long long)a.pairs * (crank + 1) / csize);
    const long long t0 = (long long)blockIdx.y * TT;
    const int tv = min(TT, (int)(a.T - t0));  // tokens of this tile

    // ---- weights of this warp's first steps are in flight while x is staged
    const bool live = rg * 16 < a.N;
    const uint8_t *wrow = a.w + (size_t)(rg >> 3) * a.kchunks * (size_t)a.chunk_bytes;
    const int w8 = rg & 7;
    auto load = [&](Step<FMT> &s, int p) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int kc = 2 * p + h;
            const bool in = live && p < p1 && kc < a.kchunks;
            const uint8_t *ch = wrow + (size_t)kc * a.chunk_bytes;
            if (BF) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    s.c[(8 * h + j) % (BF ? 16 : 4)] =
                        in ? ldg_stream(ch + ((w8 * 8 + j) * 32 + lane) * 16) : make_uint4(0, 0, 0, 0);
            } else {
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    s.c[2 * h + j] = in ? ldg_stream(ch + w8 * UNIT_BYTES + j * 512 + lane * 16) : make_uint4(0, 0, 0, 0);
                if (FMT == FMT_MXFP4) {
                    const uint2 v = in ? ldg_stream8(ch + CHUNK_MX_CODE_BYTES + (w8 * 8 + g) * 8) : make_uint2(0, 0);
                    s.s[h].x = v.x;
                    s.s[h].y = v.y;
                } else {
                    s.s[h] = in ? ldg_stream(ch + CHUNK_MX_CODE_BYTES + (w8 * 8 + g) * 16) : make_uint4(0, 0, 0, 0);
                    s.z[h] = in ? ldg_stream8(ch + CHUNK_MX_CODE_BYTES + CHUNK_I4_SCALE_BYTES + (w8 * 8 + g) * 8)
                                : make_uint2(0, 0);
                }
            }
        }
    };
    constexpr int DEPTH = BF ? 1 : 2;
    Step<FMT> st[DEPTH];
    int p = p0 + kwi;
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
        load(st[d], p + d * a.kw);

    // ---- x: this CTA's columns of the tile's tokens, as B fragments.  FP16
    // operands take x * 2^-e with e from the largest |x| of the token in these
    // columns (in [2^14, 2^15) then): exact for BF16 and E4M3 values within
    // 2^-29 of it.
    const int nvec = (p1 - p0) * 32;  // vectors of 8 values per token
    if (!BF) {
        if (tid < TT)
            xmax[tid] = 0;
        __syncthreads();
        for (int i = tid; i < tv * nvec; i += THREADS) {
            const int t = i / nvec, c = i - t * nvec;
            float v[8];
            load_x8(a, t0 + t, p0 * 256 + 8 * c, v);
            int m = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                m = max(m, __float_as_int(v[j]) & 0x7FFFFFFF);
            // nvec is a multiple of 32: a warp's lanes hold one token
            m = __reduce_max_sync(__activemask(), m);
            if (lane == 0)
                atomicMax(&xmax[t], m);
        }
        __syncthreads();
    }
    for (int i = tid; i < tv * nvec; i += THREADS) {
        const int t = i / nvec, c = i - t * nvec;
        float v[8];
        load_x8(a, t0 + t, p0 * 256 + 8 * c, v);
        uint32_t o[4];
        if (BF) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                o[j] = *reinterpret_cast<const uint32_t *>(&b);
            }
        } else {
            const int m = xmax[t];
            const int e = m == 0 ? 0 : (m >> 23) - 141;
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __half2 hh = __floats2half2_rn(scale_pow2(v[2 * j], -e), scale_pow2(v[2 * j + 1], -e));
                o[j] = *reinterpret_cast<const uint32_t *>(&hh);
                if (FMT == FMT_INT4) {
                    const float2 f = __half22float2(hh);
                    s += f.x + f.y;
                }
            }
            if (FMT == FMT_INT4) {
                // four vectors (adjacent lanes) make a block
                s += __shfl_xor_sync(__activemask(), s, 1);
                s += __shfl_xor_sync(__activemask(), s, 2);
                if ((lane & 3) == 0)
                    xsum[(c >> 2) * tv + t] = s;
            }
        }
        // values 8c .. 8c+7 of the row: k step (c & 3) / 2 of the block, low or high eight
        uint8_t *dst = xf + ((c >> 2) * tv + t) * 64 + ((c >> 1) & 1) * 8 + (c & 1) * 4;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint32_t *>(dst + j * 16) = o[j];
    }
    __syncthreads();

    // ---- weight stream
    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[n][j] = 0.f;
    // this lane's B column g: token and block (columns of tokens past tv repeat
    // the last one; nothing reads their sums)
    const int ctok = g / NB, cblk = g % NB;
    auto compute = [&](const Step<FMT> &s, int pp) {
        const uint32_t *cw = reinterpret_cast<const uint32_t *>(s.c);
        const int blk0 = (pp - p0) * 8;
#pragma unroll
        for (int grp = 0; grp < 8 / NB; ++grp) {
            float part[NT][4];
            uint4 b[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    part[n][j] = 0.f;
                const int tok = min(8 * n + ctok, tv - 1);
                b[n] = *reinterpret_cast<const uint4 *>(xf + ((blk0 + grp * NB + cblk) * tv + tok) * 64 + q * 16);
            }
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int blk = grp * NB + i;
                uint32_t a0[4], a1[4];
                if (BF) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        a0[j] = cw[(8 * blk + j) % (BF ? 64 : 16)];
                        a1[j] = cw[(8 * blk + 4 + j) % (BF ? 64 : 16)];
                    }
                } else if (FMT == FMT_MXFP4) {
                    decode_e2m1(cw[2 * blk % 16], a0);
                    decode_e2m1(cw[(2 * blk + 1) % 16], a1);
                } else {
                    decode_u4(cw[2 * blk % 16], a0);
                    decode_u4(cw[(2 * blk + 1) % 16], a1);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const bool on = NB == 1 || cblk == i;
                    mma<BF>(BF ? acc[n] : part[n], a0, on ? b[n].x : 0u, on ? b[n].y : 0u);
                    mma<BF>(BF ? acc[n] : part[n], a1, on ? b[n].z : 0u, on ? b[n].w : 0u);
                }
            }
            if (BF)
                continue;
            // scales of this lane's columns 2q, 2q+1: blocks (of this group)
            // NB = 8: 2q, 2q+1 (of both chunks); 4: 2(q&1), +1; 2: 0, 1; 1: the same block
            const int h = NB == 8 ? 0 : grp * NB / 4;  // chunk (static; NB = 8 picks by lane)
            float2 sa, sb, za = make_float2(0.f, 0.f), zb = za;
            if (FMT == FMT_MXFP4) {
                const bool hi = NB == 8 && q >= 2;
                const uint32_t ra = hi ? s.s[1].x : s.s[h].x, rb = hi ? s.s[1].y : s.s[h].y;
                // first byte of the pair inside the chunk's four
                const int sh = NB >= 4 ? 16 * (q & 1) : NB == 2 ? 16 * (grp & 1) : 16 * ((grp & 3) >> 1);
                sa = e8m0_pair(ra >> sh);
                sb = e8m0_pair(rb >> sh);
                if (NB == 1) {
                    const float fa = (grp & 1) ? sa.y : sa.x, fb = (grp & 1) ? sb.y : sb.x;
                    sa = make_float2(fa, fa);
                    sb = make_float2(fb, fb);
                }
            } else {
                const bool hi = NB == 8 && q >= 2;
                const uint4 sv = hi ? s.s[1] : s.s[h];
                const uint2 zv = hi ? s.z[1] : s.z[h];
                const bool second = NB >= 4 ? (q & 1) : NB == 2 ? (grp & 1) : ((grp & 3) >> 1);
                sa = half_pair(second ? sv.y : sv.x);
                sb = half_pair(second ? sv.w : sv.z);
                const uint32_t z0 = second ? zv.x >> 16 : zv.x, z1 = second ? zv.y >> 16 : zv.y;
                za = make_float2((float)(z0 & 255u), (float)((z0 >> 8) & 255u));
                zb = make_float2((float)(z1 & 255u), (float)((z1 >> 8) & 255u));
                if (NB == 1) {
                    const bool odd = grp & 1;
                    const float fa = odd ? sa.y : sa.x, fb = odd ? sb.y : sb.x;
                    const float ya = odd ? za.y : za.x, yb = odd ? zb.y : zb.x;
                    sa = make_float2(fa, fa), sb = make_float2(fb, fb);
                    za = make_float2(ya, ya), zb = make_float2(yb, yb);
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (FMT == FMT_MXFP4) {
                    acc[n][0] = fmaf(part[n][0], sa.x, acc[n][0]);
                    acc[n][1] = fmaf(part[n][1], sa.y, acc[n][1]);
                    acc[n][2] = fmaf(part[n][2], sb.x, acc[n][2]);
                    acc[n][3] = fmaf(part[n][3], sb.y, acc[n][3]);
                } else {
                    // sum q x - z sum x, then the group's scale
                    float xs[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int col = 2 * q + c;
                        const int tok = min(8 * n + col / NB, tv - 1);
                        xs[c] = xsum[(blk0 + grp * NB + col % NB) * tv + tok];
                    }
                    acc[n][0] = fmaf(fmaf(part[n][0], 16777216.f, -za.x * xs[0]), sa.x, acc[n][0]);
                    acc[n][1] = fmaf(fmaf(part[n][1], 16777216.f, -za.y * xs[1]), sa.y, acc[n][1]);
                    acc[n][2] = fmaf(fmaf(part[n][2], 1048576.f, -zb.x * xs[0]), sb.x, acc[n][2]);
                    acc[n][3] = fmaf(fmaf(part[n][3], 1048576.f, -zb.y * xs[1]), sb.y, acc[n][3]);
                }
            }
        }
    };
    for (; p < p1; p += DEPTH * a.kw) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            const int pp = p + d * a.kw;
            if (pp < p1)
                compute(st[d], pp);
            load(st[d], pp + DEPTH * a.kw);
        }
    }

    // ---- sums over the blocks side by side, the warps of a row group, the cluster
    const int rows = rgroups * 16;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float *o = red + (size_t)kwi * TT * rows + rwi * 16;
        if (NB == 1) {
            o[(8 * n + 2 * q) * rows + g] = acc[n][0];
            o[(8 * n + 2 * q + 1) * rows + g] = acc[n][1];
            o[(8 * n + 2 * q) * rows + g + 8] = acc[n][2];
            o[(8 * n + 2 * q + 1) * rows + g + 8] = acc[n][3];
        } else {
            float r0 = acc[n][0] + acc[n][1], r1 = acc[n][2] + acc[n][3];
            if (NB >= 4) {
                r0 += __shfl_xor_sync(0xffffffffu, r0, 1);
                r1 += __shfl_xor_sync(0xffffffffu, r1, 1);
            }
            if (NB == 8) {
                r0 += __shfl_xor_sync(0xffffffffu, r0, 2);
                r1 += __shfl_xor_sync(0xffffffffu, r1, 2);
            }
            const int tok = 2 * q / NB;  // equal values from the lanes that share a token
            o[tok * rows + g] = r0;
            o[tok * rows + g + 8] = r1;
        }
    }
    __syncthreads();
    const int total = tv * rows;
    const int row0 = tile * rows;
    for (int i = tid; i < total; i += THREADS) {
        float v = red[i];
        for (int k = 1; k < a.kw; ++k)
            v += red[(size_t)k * TT * rows + i];
        if (!BF) {
            const int m = xmax[i / rows];
            v = scale_pow2(v, m == 0 ? 0 : (m >> 23) - 141);
        }
        red[i] = v;
    }
    if (csize > 1)
        cluster_sync();
    else
        __syncthreads();
    // rank r finishes every csize-th run of THREADS sums
    for (int i = crank * THREADS + tid; i < total; i += csize * THREADS) {
        float v;
        if (csize > 1) {
            v = 0.f;
            const uint32_t local = (uint32_t)__cvta_generic_to_shared(red + i);
            for (uint32_t r = 0; r < csize; ++r) {
                uint32_t remote;
                float f;
                asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(r));
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f) : "r"(remote));
                v += f;
            }
        } else {
            v = red[i];
        }
        const int t = i / rows, n = row0 + (i - t * rows);
        if (n < a.N) {
            const long long at = (t0 + t) * a.y_ld + n;
            if (a.y_f32) {
                float *y = static_cast<float *>(a.y) + at;
                *y = a.accumulate ? *y + v : v;
            } else {
                static_cast<__nv_bfloat16 *>(a.y)[at] = __float2bfloat16_rn(v);
            }
        }
    }
    if (csize > 1)
        cluster_sync();  // a CTA's sums stay in place until every rank has read them
}

// ------------------------------------------------------------------ host side

// How a call is cut: kw warps of a CTA along K, a cluster of `cluster` CTAs
// along K, and the shared memory of a CTA.
struct Cut {
    int kw, cluster, smem, xs_off, red_off;
};

Cut cut_of(int pairs, int tt, int tv, bool i4, int kw, int cluster)
{
    Cut c;
    c.kw = kw;
    c.cluster = cluster;
    const int blocks = (pairs + cluster - 1) / cluster * 8;
    c.xs_off = blocks * tv * 64;
    c.red_off = c.xs_off + 64 + (i4 ? blocks * tv * 4 : 0);
    c.red_off = (c.red_off + 15) & ~15;
    c.smem = c.red_off + tt * WARPS * 16 * 4;
    return c;
}

constexpr int SMEM_MAX = 200 * 1024;

template <int FMT, int TB, int NT>
cudaError_t launch_linear(const LinArgs &args, cudaStream_t st)
{
    constexpr int TT = TB * NT;
    LinArgs a = args;
    const int n16 = (a.N + 15) / 16;
    const int tiles_y = (a.T + TT - 1) / TT;
    const int tv = a.T < TT ? a.T : TT;
    // warps along K first within the CTA, then over a cluster where x would not
    // fit or where the rows alone leave SMs idle
    int kw = 8, cl = 1;
    while (kw > 1 && (long long)((n16 * kw + 7) / 8) * tiles_y > 8ll * gemm::sm_count())
        kw >>= 1;
    Cut c = cut_of(a.pairs, TT, tv, FMT == FMT_INT4, kw, cl);
    while (cl < 8 &&
           (c.smem > 64 * 1024 || (long long)((n16 * kw + 7) / 8) * tiles_y * cl < 2ll * gemm::sm_count())) {
        cl *= 2;
        c = cut_of(a.pairs, TT, tv, FMT == FMT_INT4, kw, cl);
    }
    if constexpr (NT > 1) {
        if (c.smem > SMEM_MAX)  // the longest rows: fewer tokens at a time
            return launch_linear<FMT, TB, 1>(args, st);
    }
    if (c.smem > SMEM_MAX)
        return cudaErrorInvalidValue;
    a.kw = c.kw;
    a.xs_off = c.xs_off;
    a.red_off = c.red_off;
    auto kern = linear_kernel<FMT, TB, NT>;
    static std::atomic<int> attr_set[gemm::MAX_DEVICES];
    cudaError_t e = gemm::smem_limit_once(attr_set, (const void *)kern, SMEM_MAX);
    if (e != cudaSuccess)
        return e;
    const int rgroups = WARPS / c.kw;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((n16 + rgroups - 1) / rgroups * c.cluster), (unsigned)tiles_y);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = c.smem;
    cfg.stream = st;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)c.cluster;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int FMT>
cudaError_t launch_tokens(const LinArgs &a, cudaStream_t st)
{
    if constexpr (FMT != FMT_BF16) {  // (BF16 weights have no scales to apply per block)
        if (a.T == 1)
            return launch_linear<FMT, 1, 1>(a, st);
        if (a.T == 2)
            return launch_linear<FMT, 2, 1>(a, st);
        if (a.T <= 4)
            return launch_linear<FMT, 4, 1>(a, st);
    }
    return a.T <= 8 ? launch_linear<FMT, 8, 1>(a, st) : launch_linear<FMT, 8, 2>(a, st);
}

MoeStatus bad(MoeStatus s, const char *msg) { return (MoeStatus)set_last_error(s, msg); }

MoeStatus bad_cuda(const char *what, cudaError_t e)
{
    char msg[160];
    snprintf(msg, sizeof msg, "%s: %s", what, cudaGetErrorString(e));
    return bad(MOE_ECUDA, msg);
}

void destroy(MoeLinear *l)
{
    if (l->frag.base)
        cudaFree(l->frag.base);
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
    if (cudaMalloc(&f.base, f.group_bytes) != cudaSuccess) {
        cudaGetLastError();
        snprintf(msg, sizeof msg, "device allocation of %zu bytes of weights failed", f.group_bytes);
        destroy(l);
        return bad(MOE_ENOMEM, msg);
    }
    const SrcMat src = {(const uint8_t *)w->codes, (const uint8_t *)(fmt == FMT_BF16 ? nullptr : w->scales),
                        fmt == FMT_BF16 ? (long long)K * 2 : K / 2, K / 32,
                        (const uint8_t *)(fmt == FMT_INT4 ? w->zeros : nullptr)};
    if ((e = launch_repack(fmt, fmt == FMT_BF16 ? LAYOUT_FRAG : LAYOUT_FRAG_F16, false, src, src, f, 0, K, N,
                           &l->err_dev[1], st)) != cudaSuccess ||
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

size_t moe_linear_workspace_bytes(const MoeLinear *, int) { return 0; }

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
    if (ws_bytes < moe_linear_workspace_bytes(l, T))
        return bad(MOE_EWORKSPACE, "moe_linear_forward: the workspace is smaller than moe_linear_workspace_bytes");
    if ((uintptr_t)workspace % 256)
        return bad(MOE_EWORKSPACE, "moe_linear_forward: the workspace must be 256-byte aligned");
    LinArgs a{};
    a.w = l->frag.base;
    a.N = l->N;
    a.K = l->K;
    a.kchunks = l->frag.kchunks;
    a.chunk_bytes = l->frag.chunk_bytes;
    a.pairs = (a.kchunks + 1) / 2;
    a.x = x;
    a.xscales = (const uint8_t *)x_scales;
    a.x_ld = x_ld;
    a.x_mx = x_type == MOE_ROWS_MXFP8;
    a.T = T;
    a.y = y;
    a.y_ld = y_ld;
    a.y_f32 = y_type == MOE_ROWS_F32;
    a.accumulate = accumulate != 0;
    cudaStream_t st = (cudaStream_t)cuda_stream;
    const cudaError_t e = l->fmt == FMT_MXFP4  ? launch_tokens<FMT_MXFP4>(a, st)
                          : l->fmt == FMT_INT4 ? launch_tokens<FMT_INT4>(a, st)
                                               : launch_tokens<FMT_BF16>(a, st);
    if (e != cudaSuccess)
        return bad_cuda("linear layer launch", e);
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
