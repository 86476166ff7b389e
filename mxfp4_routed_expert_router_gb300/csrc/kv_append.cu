// kv_append.cu -- rotary embedding and the write into a paged key-value cache
// (moe_kv_append, include/moe.h).
//
// A row holds heads + 2 * n_kv_heads vectors of head_dim values: queries, keys, values, as the input projection leaves
// them.  Queries and keys are turned, planes (a, b) of a head's first rot_dim values by the position's angle:
//   a' = a cos - b sin,  b' = b cos + a sin
// and written as BF16 rows (queries; keys on request); keys and values go into the cache, as BF16 or as MXFP8.
//
// Bound by HBM for a prompt (each value read once and written once or twice) and by a load's latency for a few tokens.
// A thread holds 16 values of a head: with planes (i, i + rot_dim / 2) 8 values of either half, so that both of a plane
// are in one thread and every load and store has 16 bytes.  The 4 or 8 threads of a head are adjacent lanes, which
// give an MXFP8 block its largest value by shuffles.  With many tokens a thread takes the same 16 places of 4 heads, for
// which the cosines and sines (64 bytes, twice the bytes of a head's values) are loaded once.
//
// Measured (device time among other calls): one token of 56 + 16 heads of 128 1.5 us; 176 tokens of 64 + 16 heads into
// an MXFP8 cache 4.2 us; 8192 tokens of 64 + 16 heads, keys as rows too, 59 us (357 MB, 0.89 of a plain copy's rate; with
// each load waiting for the one before 74 us; 512 threads a CTA 68; 2 or 8 heads a thread 81 or 61).
//
// MXFP8 keys round once, from the exact turned value: products and sum are held as two floats (a BF16 value times a
// float leaves a float's rounding error, which an FMA gives) and the pair becomes a float rounded to odd, which no
// later rounding to four bits takes to the wrong side of a border.
#include <math.h>
#include <stdio.h>

#include <atomic>
#include <exception>
#include <map>
#include <mutex>
#include <utility>

#include "attention_internal.cuh"
#include "gemm_common.cuh"
#include "mx_encode.cuh"
#include "overlap.cuh"

namespace moe {

namespace {

__device__ int g_error;  // what a kernel recorded first since it was last taken
__device__ int g_taken;  // (a report's copy of it)

// Takes what is recorded in one step: what another stream's kernel records meanwhile comes before it or stays.
__global__ void take_error_kernel(int *flag, int *taken) { *taken = atomicExch(flag, 0); }

// Every stream hears of every error of its device: kernels do not know whose they are (a captured call's replay may run
// on any stream), and the stream that asks first must not keep an error from the one whose rows it spoilt.
struct Reports {
    std::mutex mu;
    unsigned long long count[gemm::MAX_DEVICES] = {};          // errors taken, per device
    int code[gemm::MAX_DEVICES] = {};                          // the last one
    std::map<std::pair<int, void *>, unsigned long long> seen;  // (device, stream) -> the count of its last report
};
Reports g_reports;

constexpr int THREADS = 256;

struct AppendArgs {
    const uint16_t *qkv;
    long long ld;
    int T, heads, kv, units;     // units = heads + 2 kv
    int per_token;               // threads of a token
    int tokens;                  // tokens of a CTA
    int slots_of_head;           // heads that one pass of a token's threads covers
    const int32_t *slots, *positions;
    const float *rope;
    int n_positions, rot, pairs;
    uint16_t *q_out, *k_out;
    long long q_ld, k_ld;
    void *ck, *cv;
    uint8_t *ks, *vs;
    long long n_slots;
    int page_log2;
    int *err;
};

__device__ __forceinline__ void unpack8(const uint4 &u, float v[8])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// x cos + y sin, rounded to odd where it is not a float: the products' errors are exact (FMA), the sum's by the
// two-sum of Knuth; what is left out is the rounding of their own sum, 2^-48 of the terms.
__device__ __forceinline__ float turn_odd(float x, float c, float y, float s)
{
    const float p = x * c, q = y * s;
    const float ep = fmaf(x, c, -p), eq = fmaf(y, s, -q);
    const float r = p + q, t = r - p;
    const float rest = ((p - (r - t)) + (q - t)) + (ep + eq);
    const float hi = r + rest;
    const float lo = rest - (hi - r);
    const int bits = __float_as_int(hi);
    if (lo == 0.f || (bits & 1) || !isfinite(hi) || hi == 0.f || lo != lo)
        return hi;
    return __int_as_float(bits + (((__float_as_int(lo) ^ bits) < 0) ? -1 : 1));
}

template <int D, bool MX, int HPT>
__global__ void __launch_bounds__(THREADS) kv_append_kernel(const AppendArgs a)
{
    constexpr int C = D / 16;  // threads of a head
    overlap_trigger();
    overlap_wait();
    const int idx = blockIdx.y * blockDim.x + threadIdx.x;
    const int tl = idx / a.per_token, j = idx - tl * a.per_token;
    const long long t = (long long)blockIdx.x * a.tokens + tl;
    const bool here = tl < a.tokens && t < a.T;
    const int c = j % C, hs = j / C;
    const bool turned = 16 * c < a.rot;
    // the thread's places: 8 values from `one`, 8 from `two`
    const bool halves = turned && !a.pairs;
    const int one = halves ? 8 * c : 16 * c, two = halves ? a.rot / 2 + 8 * c : 16 * c + 8;
    // all that the thread reads is asked for before anything is looked at; the cosines wait for the position alone
    uint4 u[HPT][2];
    int slot = -1, pos = 0;
    if (here) {
        pos = turned ? __ldcg(a.positions + t) : 0;
        slot = __ldcg(a.slots + t);
    }
#pragma unroll
    for (int i = 0; i < HPT; ++i) {
        const int h = hs + i * a.slots_of_head;
        u[i][0] = u[i][1] = make_uint4(0, 0, 0, 0);
        if (here && h < a.units) {
            const uint16_t *p = a.qkv + t * a.ld + (long long)h * D;
            u[i][0] = __ldcg(reinterpret_cast<const uint4 *>(p + one));
            u[i][1] = __ldcg(reinterpret_cast<const uint4 *>(p + two));
        }
    }
    float cs[8], sn[8];
    const bool known = pos >= 0 && pos < a.n_positions;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        cs[i] = sn[i] = __int_as_float(0x7FC00000);
    if (here && turned && known) {
        const float4 *p = reinterpret_cast<const float4 *>(a.rope + (long long)pos * a.rot + 8 * c);
        const float4 *q = reinterpret_cast<const float4 *>(a.rope + (long long)pos * a.rot + a.rot / 2 + 8 * c);
        const float4 c0 = __ldcg(p), c1 = __ldcg(p + 1), s0 = __ldcg(q), s1 = __ldcg(q + 1);
        cs[0] = c0.x, cs[1] = c0.y, cs[2] = c0.z, cs[3] = c0.w;
        cs[4] = c1.x, cs[5] = c1.y, cs[6] = c1.z, cs[7] = c1.w;
        sn[0] = s0.x, sn[1] = s0.y, sn[2] = s0.z, sn[3] = s0.w;
        sn[4] = s1.x, sn[5] = s1.y, sn[6] = s1.z, sn[7] = s1.w;
    }
    const bool outside = slot != -1 && (slot < 0 || slot >= a.n_slots);
    if (here && j == 0 && (outside || (slot != -1 && turned && !known)))  // (a row of padding may have any position)
        atomicCAS(a.err, 0, DEV_ERR_BOUNDS);
    if (outside)
        slot = -1;
#pragma unroll
    for (int i = 0; i < HPT; ++i) {
        const int h = hs + i * a.slots_of_head;
        const bool in = here && h < a.units;
        const bool is_v = h >= a.heads + a.kv, is_q = h < a.heads;
        const int kvh = h - a.heads - (is_v ? a.kv : 0);  // (of keys and values)
        const bool encode = MX && in && !is_q && slot >= 0;
        float v[16];
        unpack8(u[i][0], v);
        unpack8(u[i][1], v + 8);
        if (turned && !is_v) {
            float r[16];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float x = a.pairs ? v[2 * k] : v[k], y = a.pairs ? v[2 * k + 1] : v[k + 8];
                const float rx = MX && !is_q ? turn_odd(x, cs[k], -y, sn[k]) : fmaf(x, cs[k], -(y * sn[k]));
                const float ry = MX && !is_q ? turn_odd(y, cs[k], x, sn[k]) : fmaf(y, cs[k], x * sn[k]);
                r[k] = rx;
                r[k + 8] = ry;
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                v[k] = a.pairs ? r[(k & 1) * 8 + k / 2] : r[k];
                v[k + 8] = a.pairs ? r[(k & 1) * 8 + 4 + k / 2] : r[k + 8];
            }
        }
        if (in && (is_q ? a.q_out != nullptr : !is_v && a.k_out != nullptr)) {
            uint16_t *o = is_q ? a.q_out + t * a.q_ld + (long long)h * D : a.k_out + t * a.k_ld + (long long)kvh * D;
            *reinterpret_cast<uint4 *>(o + one) = bf16x8(v);
            *reinterpret_cast<uint4 *>(o + two) = bf16x8(v + 8);
        }
        const long long at = in && !is_q && slot >= 0
                                 ? (((long long)(slot >> a.page_log2) * a.kv + kvh) << a.page_log2) +
                                       (slot & ((1 << a.page_log2) - 1))
                                 : 0;  // row of the cache
        if (!MX) {
            if (in && !is_q && slot >= 0) {
                uint16_t *o = static_cast<uint16_t *>(is_v ? a.cv : a.ck) + at * D;
                *reinterpret_cast<uint4 *>(o + one) = bf16x8(v);
                *reinterpret_cast<uint4 *>(o + two) = bf16x8(v + 8);
            }
        } else if (__any_sync(0xffffffffu, encode)) {
            float m1 = 0.f, m2 = 0.f;  // the largest of either 8 values
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                m1 = fmaxf(m1, fabsf(v[k]));
                m2 = fmaxf(m2, fabsf(v[k + 8]));
            }
            int byte1 = 0, byte2 = 0;
#pragma unroll
            for (int b = 0; b < D / 32; ++b) {
                float m = fmaxf(one / 32 == b ? m1 : 0.f, two / 32 == b ? m2 : 0.f);
#pragma unroll
                for (int o = C / 2; o > 0; o >>= 1)
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                const int byte = mx_scale_byte(m);
                byte1 = one / 32 == b ? byte : byte1;
                byte2 = two / 32 == b ? byte : byte2;
                if (encode && c == b)  // (C >= D / 32 threads a head: one for each block)
                    (is_v ? a.vs : a.ks)[at * (D / 32) + b] = (uint8_t)byte;
            }
            if (encode) {
                uint8_t *o = static_cast<uint8_t *>(is_v ? a.cv : a.ck) + at * D;
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const float mul = __int_as_float((254 - (p ? byte2 : byte1)) << 23);  // 2^(127 - byte): exact
                    float *w = v + 8 * p;
#pragma unroll
                    for (int k = 0; k < 8; ++k)  // the conversion saturates an infinity; here it is NaN
                        w[k] = isinf(w[k]) ? __int_as_float(0x7FC00000) : w[k] * mul;
                    *reinterpret_cast<uint2 *>(o + (p ? two : one)) =
                        make_uint2(e4m3x2(w[0], w[1]) | e4m3x2(w[2], w[3]) << 16,
                                   e4m3x2(w[4], w[5]) | e4m3x2(w[6], w[7]) << 16);
                }
            }
        }
    }
}

template <int D, bool MX>
cudaError_t launch_append(AppendArgs &a, cudaStream_t st)
{
    constexpr int C = D / 16, MANY = 4;
    const bool many = (long long)a.T * a.units * C >= 2048ll * gemm::sm_count();
    a.slots_of_head = many ? (a.units + MANY - 1) / MANY : a.units;
    a.per_token = a.slots_of_head * C;
    a.tokens = a.per_token >= THREADS ? 1 : THREADS / a.per_token;
    const int n = a.per_token * a.tokens, threads = n >= THREADS ? THREADS : (n + 31) & ~31;
    const dim3 grid((unsigned)((a.T + a.tokens - 1) / a.tokens), (unsigned)((n + threads - 1) / threads));
    return many ? launch_overlapped(kv_append_kernel<D, MX, MANY>, grid, threads, 0, 1, st, a)
                : launch_overlapped(kv_append_kernel<D, MX, 1>, grid, threads, 0, 1, st, a);
}

MoeStatus bad(MoeStatus s, const char *msg) { return (MoeStatus)set_last_error(s, msg); }

}  // namespace

cudaError_t attention_error_flag(int **flag)
{
    static std::atomic<int *> cached[gemm::MAX_DEVICES];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= gemm::MAX_DEVICES)
        return cudaErrorInvalidDevice;
    if (!(*flag = cached[dev].load(std::memory_order_acquire))) {
        void *p = nullptr;
        if ((e = cudaGetSymbolAddress(&p, g_error)) != cudaSuccess)
            return e;
        cached[dev].store(*flag = static_cast<int *>(p), std::memory_order_release);
    }
    return cudaSuccess;
}

MoeStatus check_kv_cache(const MoeKvCache *c)
{
    char msg[160];
    if (!c)
        return bad(MOE_EINVAL, "key-value cache: NULL");
    if (c->type != MOE_ROWS_BF16 && c->type != MOE_ROWS_MXFP8)
        return bad(MOE_EINVAL, "key-value cache: BF16 or MXFP8 rows are needed");
    if (c->head_dim != 64 && c->head_dim != 128) {
        snprintf(msg, sizeof msg, "key-value cache: head_dim (%d) must be 64 or 128", c->head_dim);
        return bad(MOE_EDIMS, msg);
    }
    if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1))) {
        snprintf(msg, sizeof msg, "key-value cache: page_size (%d) must be a power of two in 16 .. 256", c->page_size);
        return bad(MOE_EDIMS, msg);
    }
    if (c->n_kv_heads < 1 || c->n_kv_heads > ATTN_MAX_HEADS)
        return bad(MOE_EINVAL, "key-value cache: n_kv_heads out of range [1, 1024]");
    if (c->n_pages < 1 || (long long)c->n_pages * c->page_size > 0x7FFFFFFFll)
        return bad(MOE_EINVAL, "key-value cache: 1 page or more, and fewer than 2^31 rows, are needed");
    if (!c->k || !c->v || (uintptr_t)c->k % 16 || (uintptr_t)c->v % 16)
        return bad(MOE_EINVAL, "key-value cache: k and v must be given and 16-byte aligned");
    if (c->type == MOE_ROWS_MXFP8 &&
        (!c->k_scales || !c->v_scales || (uintptr_t)c->k_scales % 16 || (uintptr_t)c->v_scales % 16))
        return bad(MOE_EINVAL, "key-value cache: MXFP8 needs k_scales and v_scales, 16-byte aligned");
    return MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" MoeStatus moe_kv_append(const MoeKvCache *cache, const void *qkv, long long qkv_ld, int T, int n_heads,
                                   const int32_t *slots, const int32_t *positions, const float *rope, int n_positions,
                                   int rot_dim, MoeRope style, void *q_out, long long q_ld, void *k_out,
                                   long long k_ld, void *cuda_stream)
{
    char msg[160];
    const MoeStatus s = check_kv_cache(cache);
    if (s != MOE_OK)
        return s;
    const int D = cache->head_dim, kv = cache->n_kv_heads;
    if (T < 0 || T > (1 << 24)) {
        snprintf(msg, sizeof msg, "T = %d out of range [0, 2^24]", T);
        return bad(MOE_EINVAL, msg);
    }
    if (n_heads < 1 || n_heads > ATTN_MAX_HEADS)
        return bad(MOE_EINVAL, "moe_kv_append: n_heads out of range [1, 1024]");
    if (style != MOE_ROPE_HALVES && style != MOE_ROPE_PAIRS)
        return bad(MOE_EINVAL, "moe_kv_append: unknown rotation style");
    if (rope && (rot_dim < 16 || rot_dim % 16 || rot_dim > D || n_positions < 1)) {
        snprintf(msg, sizeof msg, "moe_kv_append: rot_dim (%d) must be a multiple of 16 in 16 .. head_dim, n_positions "
                                  "(%d) at least 1", rot_dim, n_positions);
        return bad(MOE_EDIMS, msg);
    }
    if (T == 0)
        return MOE_OK;
    if (!qkv || !slots || (rope && !positions))
        return bad(MOE_EINVAL, "moe_kv_append: NULL qkv, slots, or positions of a rotation");
    const long long w = (long long)(n_heads + 2 * kv) * D;
    if (qkv_ld < w || (q_out && q_ld < (long long)n_heads * D) || (k_out && k_ld < (long long)kv * D))
        return bad(MOE_EINVAL, "moe_kv_append: a row stride is below the row's values");
    if (!rows_16b(qkv, qkv_ld) || (q_out && !rows_16b(q_out, q_ld)) || (k_out && !rows_16b(k_out, k_ld)) ||
        (rope && (uintptr_t)rope % 16) || (uintptr_t)slots % 4 || (uintptr_t)positions % 4)
        return bad(MOE_EINVAL, "moe_kv_append: rows and rope must start on 16-byte boundaries, slots and positions on "
                               "4-byte ones");
    AppendArgs a{};
    cudaError_t e = attention_error_flag(&a.err);
    if (e == cudaSuccess) {
        a.qkv = static_cast<const uint16_t *>(qkv);
        a.ld = qkv_ld;
        a.T = T;
        a.heads = n_heads;
        a.kv = kv;
        a.units = n_heads + 2 * kv;
        a.slots = slots;
        a.positions = positions;
        a.rope = rope;
        a.n_positions = n_positions;
        a.rot = rope ? rot_dim : 0;
        a.pairs = style == MOE_ROPE_PAIRS;
        a.q_out = static_cast<uint16_t *>(q_out);
        a.q_ld = q_ld;
        a.k_out = static_cast<uint16_t *>(k_out);
        a.k_ld = k_ld;
        a.ck = cache->k;
        a.cv = cache->v;
        a.ks = static_cast<uint8_t *>(cache->k_scales);
        a.vs = static_cast<uint8_t *>(cache->v_scales);
        a.n_slots = (long long)cache->n_pages * cache->page_size;
        while ((1 << a.page_log2) < cache->page_size)
            ++a.page_log2;
        cudaStream_t st = (cudaStream_t)cuda_stream;
        const bool mx = cache->type == MOE_ROWS_MXFP8;
        if (D == 128)
            e = mx ? launch_append<128, true>(a, st) : launch_append<128, false>(a, st);
        else
            e = mx ? launch_append<64, true>(a, st) : launch_append<64, false>(a, st);
    }
    if (e != cudaSuccess) {
        snprintf(msg, sizeof msg, "key-value append launch: %s", cudaGetErrorString(e));
        return bad(MOE_ECUDA, msg);
    }
    return MOE_OK;
}

extern "C" MoeStatus moe_attention_status(void *cuda_stream)
{
    char msg[160];
    cudaStream_t st = (cudaStream_t)cuda_stream;
    int *flag = nullptr, dev = 0, got = 0;
    cudaError_t e = attention_error_flag(&flag);
    if (e == cudaSuccess)
        e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaStreamSynchronize(st);
    try {
        std::lock_guard<std::mutex> lock(g_reports.mu);
        unsigned long long &seen = g_reports.seen[{dev, cuda_stream}];
        void *taken = nullptr;
        if (e == cudaSuccess)
            e = cudaGetSymbolAddress(&taken, g_taken);
        if (e == cudaSuccess) {
            cudaLaunchConfig_t cfg{};
            cfg.gridDim = cfg.blockDim = 1;
            cfg.stream = st;
            e = cudaLaunchKernelEx(&cfg, take_error_kernel, flag, static_cast<int *>(taken));
        }
        if (e == cudaSuccess)
            e = cudaMemcpyAsync(&got, taken, sizeof got, cudaMemcpyDeviceToHost, st);
        if (e == cudaSuccess)
            e = cudaStreamSynchronize(st);
        if (e == cudaSuccess) {
            if (got) {
                ++g_reports.count[dev];
                g_reports.code[dev] = got;
            }
            got = seen != g_reports.count[dev] ? g_reports.code[dev] : 0;
            seen = g_reports.count[dev];
        }
    } catch (const std::exception &x) {
        snprintf(msg, sizeof msg, "moe_attention_status: %s", x.what());
        return bad(MOE_ENOMEM, msg);
    }
    if (e != cudaSuccess) {
        snprintf(msg, sizeof msg, "moe_attention_status: %s", cudaGetErrorString(e));
        return bad(MOE_ECUDA, msg);
    }
    if (got) {
        snprintf(msg, sizeof msg, "attention: a kernel reported device error %d", got);
        return bad(MOE_EDEVICE, msg);
    }
    return MOE_OK;
}
