// norm.cu -- residual addition and RMS norm in front of the layer's operators
// (moe_add_rmsnorm, include/moe.h): BF16 rows for the experts and the router,
// MXFP8 rows for the linear layers.
//
//   s = round(residual + delta),  n = s * (gain / sqrt(mean(s^2) + eps)),
//   y = bf16(n),  q = e4m3(n * 2^-p) with p per 32 values.
//
// One pass over the data: a row stays in registers between the sum of squares
// and the outputs, so that a value is read once and written once per output.
// Bound by HBM for many rows and by one load's latency, the row's reduction and
// the stores for one token.  A thread holds vectors of 8 values (one or two
// 16-byte loads); the four lanes of a 32-value MXFP8 block are adjacent, so its
// largest value takes two shuffles.  One CTA per row, as many threads as the row
// has vectors (up to 1024, then two, four or eight vectors a thread): a row of 7168
// is 28 warps of one vector each, two rows to an SM.
//
// Measured, FP32 residual and delta, sum, y and q: 8192 rows of 7168 values 128 us
// (882 MB, 6.9 TB/s: the rate of a plain copy), of BF16 94 us (529 MB, 5.6 TB/s: the
// instructions show); 176 rows 5.9 us from HBM, 5.2 from L2; one row of BF16 2.5 us, launch
// included.  Above 32768 values a thread's eight vectors do not fit 64 registers: 120 to
// 476 bytes are spilled (64 rows of 40960 BF16 values: 14.7 us, 24 MB).
#include <math.h>
#include <stdio.h>

#include "../../include/moe.h"
#include "moe_internal.cuh"
#include "mx_encode.cuh"
#include "overlap.cuh"

namespace moe {

namespace {

struct NormArgs {
    const void *res, *delta;
    long long res_ld, delta_ld;
    const void *gain;
    int gain_type;
    float eps;
    int H;
    void *sum;
    long long sum_ld;
    uint16_t *y;
    long long y_ld;
    uint8_t *q;
    long long q_ld;
    uint8_t *qs;
};

// 8 consecutive values from element `at` (16-byte aligned) of a row.  Plain
// loads, not the read-only path: sum may be written in place of the input.
template <int TYPE>
__device__ __forceinline__ void load8(const void *p, long long at, float v[8])
{
    if (TYPE == MOE_ROWS_BF16) {
        const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + at);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
        const float4 a = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at);
        const float4 b = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at + 4);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
}

// One row per CTA, VPT vectors of 8 values per thread.  RES and DELTA are row
// types (DELTA -1: none).
template <int RES, int DELTA, int VPT>
__global__ void __launch_bounds__(1024) add_rmsnorm_kernel(const NormArgs a)
{
    __shared__ float red[32];
    const int tid = threadIdx.x, lane = tid & 31;
    const int nv = a.H / 8;
    const long long t = blockIdx.x;
    overlap_wait();
    float v[VPT][8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = tid + i * (int)blockDim.x;
        if (c < nv) {
            load8<RES>(a.res, t * a.res_ld + 8 * c, v[i]);
            if (DELTA >= 0) {
                float d[8];
                load8<DELTA>(a.delta, t * a.delta_ld + 8 * c, d);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[i][j] += d[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[i][j] = 0.f;
        }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = tid + i * (int)blockDim.x;
        const bool in = c < nv;
        if (RES == MOE_ROWS_BF16 && DELTA >= 0) {
            // the norm is that of what the stream holds
            const uint4 u = bf16x8(v[i]);
            if (in && a.sum)
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.sum) + t * a.sum_ld + 8 * c) = u;
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[i][2 * j] = __uint_as_float(w[j] << 16);
                v[i][2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
            }
        } else if (in && a.sum) {
            if (RES == MOE_ROWS_BF16) {
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.sum) + t * a.sum_ld + 8 * c) = bf16x8(v[i]);
            } else {
                float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(a.sum) + t * a.sum_ld + 8 * c);
                o[0] = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
                o[1] = make_float4(v[i][4], v[i][5], v[i][6], v[i][7]);
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            ss = fmaf(v[i][j], v[i][j], ss);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
    overlap_trigger();
    const int nw = blockDim.x >> 5;  // warps of a row
    if (nw > 1) {
        if (lane == 0)
            red[tid >> 5] = ss;
        __syncthreads();
        ss = lane < nw ? red[lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
    if (!a.y && !a.q)
        return;
    // 1 / sqrt(x) as hi + lo (one Newton step, whose residual 1 - x hi^2 is taken
    // exactly), so that n below rounds once: an E4M3 value next to a border falls on
    // the side that the formula gives, but for the error of the mean
    const float x = ss / (float)a.H + a.eps;
    const float hi = rsqrtf(x);
    const float xh = x * hi;
    float lo = 0.5f * hi * (fmaf(-xh, hi, 1.f) - fmaf(x, hi, -xh) * hi);
    lo = isfinite(lo) ? lo : 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = tid + i * (int)blockDim.x;
        const bool in = c < nv;
        float g[8];
        if (a.gain && in) {
            if (a.gain_type == MOE_ROWS_BF16)
                load8<MOE_ROWS_BF16>(a.gain, 8 * c, g);
            else
                load8<MOE_ROWS_F32>(a.gain, 8 * c, g);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                g[j] = 1.f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float p = v[i][j] * hi;
            const float rest = fmaf(v[i][j], lo, fmaf(v[i][j], hi, -p));
            v[i][j] = fmaf(p, g[j], rest * g[j]);
        }
        if (in && a.y)
            *reinterpret_cast<uint4 *>(a.y + t * a.y_ld + 8 * c) = bf16x8(v[i]);
        if (a.q) {
            float m = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                m = fmaxf(m, fabsf(v[i][j]));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
            const int byte = mx_scale_byte(m);
            const float mul = __int_as_float((254 - byte) << 23);  // 2^(127 - byte): exact
#pragma unroll
            for (int j = 0; j < 8; ++j)  // the conversion saturates an infinity; here it is NaN
                v[i][j] = isinf(v[i][j]) ? __int_as_float(0x7FC00000) : v[i][j] * mul;
            if (in) {
                *reinterpret_cast<uint2 *>(a.q + t * a.q_ld + 8 * c) =
                    make_uint2(e4m3x2(v[i][0], v[i][1]) | e4m3x2(v[i][2], v[i][3]) << 16,
                               e4m3x2(v[i][4], v[i][5]) | e4m3x2(v[i][6], v[i][7]) << 16);
                if ((lane & 3) == 0)
                    a.qs[t * (a.H / 32) + c / 4] = (uint8_t)byte;
            }
        }
    }
}

template <int RES, int DELTA>
cudaError_t launch_norm(const NormArgs &a, int T, cudaStream_t st)
{
    const int nv = a.H / 8;
    const int vpt = nv <= 1024 ? 1 : nv <= 2048 ? 2 : nv <= 4096 ? 4 : 8;
    const int threads = ((nv + vpt - 1) / vpt + 31) & ~31;
    switch (vpt) {
    case 1: return launch_overlapped(add_rmsnorm_kernel<RES, DELTA, 1>, T, threads, 0, 1, st, a);
    case 2: return launch_overlapped(add_rmsnorm_kernel<RES, DELTA, 2>, T, threads, 0, 1, st, a);
    case 4: return launch_overlapped(add_rmsnorm_kernel<RES, DELTA, 4>, T, threads, 0, 1, st, a);
    default: return launch_overlapped(add_rmsnorm_kernel<RES, DELTA, 8>, T, threads, 0, 1, st, a);
    }
}

bool rows_aligned(const void *p, long long ld, int size) { return (uintptr_t)p % 16 == 0 && ld * size % 16 == 0; }

MoeStatus bad(MoeStatus s, const char *msg) { return (MoeStatus)set_last_error(s, msg); }

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" MoeStatus moe_add_rmsnorm(const void *residual, MoeRowType residual_type, long long residual_ld,
                                     const void *delta, MoeRowType delta_type, long long delta_ld, const void *gain,
                                     MoeRowType gain_type, float eps, int T, int H, void *sum, long long sum_ld,
                                     void *y, long long y_ld, void *q, long long q_ld, void *q_scales,
                                     void *cuda_stream)
{
    char msg[160];
    if (T < 0 || T > (1 << 24)) {
        snprintf(msg, sizeof msg, "T = %d out of range [0, 2^24]", T);
        return bad(MOE_EINVAL, msg);
    }
    if (H < 32 || H % 32 || H > 65536) {
        snprintf(msg, sizeof msg, "H (%d) must be a multiple of 32 in 32 .. 65536", H);
        return bad(MOE_EDIMS, msg);
    }
    if ((residual_type != MOE_ROWS_BF16 && residual_type != MOE_ROWS_F32) ||
        (delta && delta_type != MOE_ROWS_BF16 && delta_type != MOE_ROWS_F32) ||
        (gain && gain_type != MOE_ROWS_BF16 && gain_type != MOE_ROWS_F32))
        return bad(MOE_EINVAL, "moe_add_rmsnorm: residual, delta and gain are BF16 or F32");
    if (!(eps >= 0.f) || isinf(eps))
        return bad(MOE_EINVAL, "moe_add_rmsnorm: eps must be finite and not negative");
    if (T == 0)
        return MOE_OK;
    if (!residual || (!sum && !y && !q))
        return bad(MOE_EINVAL, "moe_add_rmsnorm: NULL residual, or no output");
    if (q && !q_scales)
        return bad(MOE_EINVAL, "moe_add_rmsnorm: q without q_scales");
    if (residual_ld < H || (delta && delta_ld < H) || (sum && sum_ld < H) || (y && y_ld < H) || (q && q_ld < H))
        return bad(MOE_EINVAL, "moe_add_rmsnorm: a row stride is below H");
    const int rs = residual_type == MOE_ROWS_F32 ? 4 : 2, ds = delta_type == MOE_ROWS_F32 ? 4 : 2;
    if (!rows_aligned(residual, residual_ld, rs) || (delta && !rows_aligned(delta, delta_ld, ds)) ||
        (sum && !rows_aligned(sum, sum_ld, rs)) || (y && !rows_aligned(y, y_ld, 2)) ||
        (q && !rows_aligned(q, q_ld, 1)) || (gain && (uintptr_t)gain % 16))
        return bad(MOE_EINVAL, "moe_add_rmsnorm: rows and gain must start on 16-byte boundaries");
    NormArgs a{};
    a.res = residual;
    a.res_ld = residual_ld;
    a.delta = delta;
    a.delta_ld = delta_ld;
    a.gain = gain;
    a.gain_type = gain_type;
    a.eps = eps;
    a.H = H;
    a.sum = sum;
    a.sum_ld = sum_ld;
    a.y = (uint16_t *)y;
    a.y_ld = y_ld;
    a.q = (uint8_t *)q;
    a.q_ld = q_ld;
    a.qs = (uint8_t *)q_scales;
    cudaStream_t st = (cudaStream_t)cuda_stream;
    constexpr int B = MOE_ROWS_BF16, F = MOE_ROWS_F32;
    const int d = delta ? (int)delta_type : -1;
    cudaError_t e;
    if (residual_type == MOE_ROWS_BF16)
        e = d < 0 ? launch_norm<B, -1>(a, T, st) : d == B ? launch_norm<B, B>(a, T, st) : launch_norm<B, F>(a, T, st);
    else
        e = d < 0 ? launch_norm<F, -1>(a, T, st) : d == B ? launch_norm<F, B>(a, T, st) : launch_norm<F, F>(a, T, st);
    if (e != cudaSuccess) {
        snprintf(msg, sizeof msg, "RMS norm launch: %s", cudaGetErrorString(e));
        return bad(MOE_ECUDA, msg);
    }
    return MOE_OK;
}
