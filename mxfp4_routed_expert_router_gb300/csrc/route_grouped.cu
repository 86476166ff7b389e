// route_grouped.cu -- group-limited routing (moe_route_grouped,
// include/moe.h): scores s = sigmoid(l) or softmax(l), keys c = s + bias, the
// k_groups best groups of consecutive experts, the k largest keys among them,
// weights from the scores.
//
// One warp per token.  A group's experts are spread over LG lanes, the largest
// power of two with n_groups * LG <= 32, so that a lane serves one group and a
// group's score is a shuffle reduction inside those lanes: lane = LG * group +
// sub holds the keys of experts group * GS + sub + LG * i, i < NV.  Keys are
// held as order keys (unsigned order = the selection's order; 0 is "switched
// off, or taken", 1 is NaN).
//
// The selection is that of FP64 keys, computed in FP32 wherever that is enough.
// With keys within an error e of the FP64 ones, an order whose neighbours lie
// more than 2 e apart is the FP64 order.  So route_fast selects on FP32 keys and
// measures the gaps that its result rests on (after the last group that stays;
// after each kept key); a row with a gap too small, equal keys or a value that is
// not finite is done again on FP64 keys (route_exact).  Where only the order of
// the kept keys is in doubt, FP64 keys of the experts that can be among them, one a
// lane, decide it: a row in route_exact takes several us, which a call of thousands
// of rows would wait for at its end.  The errors, with u = 2^-24:
//   sigmoid: exp 2 ulp (4 u), addition and division (2 u): below 8 u of the score
//   softmax: exp 4 u; its argument l - max rounded, |l - max| u (below 76 u for the
//     scores above 1e-30 taken here; times exp(l - max), below 0.37 u of the
//     largest); the sum of at most 64 terms a lane and 5 shuffles (69 u) of terms
//     off by 4 u and on average |l - max| < 7 u; the division u: below 96 u of the
//     row's largest score.  The sum is the same for every expert and turns no order
//     around: without a bias a key counts as off by (5 + |l - max|) u of itself, with
//     |l - max| from the key (err_of takes 8 + 1.1 |log|, which also holds for the sum
//     of two keys: e |log e| of the lesser is below the greater's, or below 0.37)
//   key with a bias: the score's, and u |key| for the addition
// Without a bias the error is relative to the key, with one it is taken from the
// row's largest score (ABS) and key.
// Where the order of groups is in doubt, the same is done for the experts that can
// make up the scores of the groups between the border's error bounds.
// Issue bound for many rows (a row is 4 E bytes), latency bound for few: all of a
// row's loads come before its arithmetic.  Sigmoid scores with a bias, k = 8, 256
// experts in 8 groups, 4 kept: 8192 rows 17 us (1.3 us of HBM time; FP64 keys for every
// row took 147 us, for the whole of each unsure row up to 28 us); 176 rows 4.5 us; one
// row 4.5 us (FP64: 15 us).
#include <math.h>
#include <stdio.h>

#include "../../include/moe.h"
#include "moe_internal.cuh"
#include "overlap.cuh"

namespace moe {

namespace {

typedef unsigned long long u64;

// Four rows a CTA: of 32 to 256 threads, 128 were the fastest or as fast as any
// (1024 rows of 256 experts 6.1 us against 7.0 with 256; 8192 rows the same).
constexpr int ROUTE_THREADS = 128;

struct RouteArgs {
    const float *logits, *bias;
    int T, E, k, n_groups, k_groups;
    int gs, lg;  // experts of a group, lanes of a group
    int top2, renorm;
    float scale;
    int *ids;
    float *w;
};

// unsigned order of a real's value: +0 and -0 equal, NaN = 1 below every number
__device__ __forceinline__ u64 order_key(double d)
{
    if (isnan(d))
        return 1ull;
    if (d == 0.0)
        d = 0.0;
    const u64 b = (u64)__double_as_longlong(d);
    return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

__device__ __forceinline__ double key_value(u64 k)
{
    if (k <= 1ull)
        return k ? __longlong_as_double(0x7FF8000000000000ll) : -INFINITY;
    return __longlong_as_double((long long)((k >> 63) ? (k & 0x7FFFFFFFFFFFFFFFull) : ~k));
}

__device__ __forceinline__ u64 warp_max(u64 m)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const u64 other = __shfl_xor_sync(0xffffffffu, m, o);
        m = other > m ? other : m;
    }
    return m;
}

// One row on FP64 keys (a whole warp).
template <int SCORE, int NV>
__device__ __noinline__ void route_exact(const RouteArgs &a, long long t)
{
    const int lane = threadIdx.x & 31;
    const float *row = a.logits + t * a.E;
    const int grp = lane / a.lg, sub = lane - grp * a.lg;
    const bool has_grp = grp < a.n_groups;

    // softmax: the row's largest logit (NaN ignored) and the sum of exponentials
    double mx = 0.0, sum = 1.0;
    if (SCORE == MOE_SCORE_SOFTMAX) {
        float m = -INFINITY;
        for (int e = lane; e < a.E; e += 32)
            m = fmaxf(m, row[e]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        mx = (double)m;
        sum = 0.0;
        for (int e = lane; e < a.E; e += 32)
            if (row[e] != -INFINITY)
                sum += exp((double)row[e] - mx);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    auto score = [&](float l) {
        return SCORE == MOE_SCORE_SOFTMAX ? exp((double)l - mx) / sum : 1.0 / (1.0 + exp(-(double)l));
    };

    u64 key[NV];
    u64 b1 = 0ull, b2 = 0ull;  // the lane's two largest keys
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = sub + a.lg * i;
        key[i] = 0ull;
        if (has_grp && j < a.gs) {
            const int e = grp * a.gs + j;
            const float l = row[e];
            if (l != -INFINITY)
                key[i] = order_key(score(l) + (a.bias ? (double)a.bias[e] : 0.0));
        }
        b2 = max(b2, min(b1, key[i]));
        b1 = max(b1, key[i]);
    }

    if (a.k_groups < a.n_groups) {
        for (int o = 1; o < a.lg; o <<= 1) {
            const u64 o1 = __shfl_xor_sync(0xffffffffu, b1, o), o2 = __shfl_xor_sync(0xffffffffu, b2, o);
            b2 = max(max(b2, o2), min(b1, o1));
            b1 = max(b1, o1);
        }
        // a group's score, in each of its lanes; a group with every expert off keeps 0
        u64 gk = b1;
        if (a.top2 && b2 != 0ull)
            gk = order_key(key_value(b1) + key_value(b2));
        bool kept = false;
        for (int r = 0; r < a.k_groups; ++r) {
            const u64 mine = has_grp && !kept ? gk : 0ull;
            const u64 m = warp_max(mine);
            const unsigned g = __reduce_min_sync(0xffffffffu, mine == m && has_grp && !kept ? (unsigned)grp : 64u);
            kept = kept || (unsigned)grp == g;
        }
        if (!kept)
#pragma unroll
            for (int i = 0; i < NV; ++i)
                key[i] = 0ull;
    }

    int my_e = -1;
    for (int j = 0; j < a.k; ++j) {
        u64 best = 0ull;
        int bi = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (key[i] > best) {  // strict: the lowest expert of the lane among equals
                best = key[i];
                bi = i;
            }
        const u64 m = warp_max(best);
        if (m == 0ull)
            break;  // no expert is left: empty slots
        const unsigned mine = (unsigned)(grp * a.gs + sub + a.lg * bi);
        const unsigned e = __reduce_min_sync(0xffffffffu, best == m ? mine : 0xFFFFFFFFu);
        if (mine == e) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (i == bi)
                    key[i] = 0ull;
        }
        if (lane == j)
            my_e = (int)e;
    }
    double s = my_e >= 0 ? score(row[my_e]) : 0.0;
    if (a.renorm) {
        double tot = s;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            tot += __shfl_xor_sync(0xffffffffu, tot, o);
        s = tot == 0.0 ? 0.0 : s / tot;
    }
    if (lane < a.k) {
        a.ids[t * a.k + lane] = my_e;
        a.w[t * a.k + lane] = my_e >= 0 ? (float)((double)a.scale * s) : 0.f;
    }
}

// FP32 order keys: unsigned order of finite values, 0 is below all of them
__device__ __forceinline__ uint32_t order_key32(float f)
{
    const uint32_t b = __float_as_uint(f + 0.f);  // (-0 becomes +0)
    return (b >> 31) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float key_value32(uint32_t k)
{
    return k ? __uint_as_float((k >> 31) ? (k & 0x7FFFFFFFu) : ~k) : -INFINITY;
}

// One row on FP32 keys (a whole warp; cand: 32 ints of its own in shared memory):
// writes the row and returns true when the selection is certain.
template <int SCORE, int NV>
__device__ __forceinline__ bool route_fast(const RouteArgs &a, long long t, int *cand)
{
    constexpr float U = 5.9604645e-8f;  // 2^-24
    constexpr float REL = 8.f * U;
    constexpr float ABS = (SCORE == MOE_SCORE_SOFTMAX ? 96.f : 8.f) * U;
    const int lane = threadIdx.x & 31;
    const float *row = a.logits + t * a.E;
    const int grp = lane / a.lg, sub = lane - grp * a.lg;
    const bool has_grp = grp < a.n_groups;
    const float *mine = row + grp * a.gs + sub;

    float l[NV], bias[NV];  // every load before the first use
#pragma unroll
    for (int i = 0; i < NV; ++i)
        l[i] = has_grp && sub + a.lg * i < a.gs ? mine[a.lg * i] : -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        bias[i] = a.bias && has_grp && sub + a.lg * i < a.gs ? a.bias[grp * a.gs + sub + a.lg * i] : 0.f;
    u64 on = 0ull;          // bit i: expert i of the lane is not switched off
#pragma unroll
    for (int i = 0; i < NV; ++i)
        on |= (u64)(l[i] != -INFINITY) << i;
    float mx = 0.f, inv = 1.f;
    if (SCORE == MOE_SCORE_SOFTMAX) {
        mx = l[0];
#pragma unroll
        for (int i = 1; i < NV; ++i)
            mx = fmaxf(mx, l[i]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            l[i] = expf(l[i] - mx);  // switched off: 0 (mx is a number), or NaN (every expert is off)
            sum += l[i];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
        inv = sum;
    }
    uint32_t key[NV];
    uint32_t b1 = 0u, b2 = 0u;          // the lane's two largest keys
    float smax = 0.f, kmax = 0.f;       // largest score and |key|
    bool fine = true;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const bool is_on = on >> i & 1;
        // (a division of zero or by an infinity would take the slow path for the whole warp)
        const float v = is_on ? l[i] : SCORE == MOE_SCORE_SOFTMAX ? inv : 0.f;
        const float sc = SCORE == MOE_SCORE_SOFTMAX ? v / inv : 1.f / (1.f + expf(-v));
        const float c = sc + bias[i];
        // (a score below FP32's normal range has no relative accuracy)
        fine = fine && (!is_on || (isfinite(c) && sc > 1e-30f));
        smax = fmaxf(smax, is_on ? sc : 0.f);
        kmax = fmaxf(kmax, is_on ? fabsf(c) : 0.f);
        key[i] = is_on ? order_key32(c) : 0u;
        b2 = max(b2, min(b1, key[i]));
        b1 = max(b1, key[i]);
    }
    if (!__all_sync(0xffffffffu, fine))
        return false;
    // twice the error of a key, absolute: with a bias the same for every key
    const uint32_t sm = __reduce_max_sync(0xffffffffu, __float_as_uint(smax));
    const uint32_t km = __reduce_max_sync(0xffffffffu, __float_as_uint(kmax));
    const float err2 = 2.f * (ABS * __uint_as_float(sm) + U * __uint_as_float(km));
    auto err_of = [&](float c) {
        if (a.bias)
            return err2;
        return SCORE == MOE_SCORE_SOFTMAX ? 2.f * U * c * (8.f + 1.1f * fabsf(__logf(c * inv))) : 2.f * REL * c;
    };

    // FP64 keys of up to 32 experts, one a lane (a warp's work; 0 for lanes without one)
    auto keys64 = [&](int e, bool has) {
        double sum64 = 0.0;
        if (SCORE == MOE_SCORE_SOFTMAX) {
#pragma unroll 1
            for (int i = 0; i < NV; ++i)
                if (has_grp && sub + a.lg * i < a.gs && mine[a.lg * i] != -INFINITY)
                    sum64 += exp((double)mine[a.lg * i] - (double)mx);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                sum64 += __shfl_xor_sync(0xffffffffu, sum64, o);
        }
        if (!has)
            return (u64)0;
        const double l64 = (double)row[e];
        const double s64 = SCORE == MOE_SCORE_SOFTMAX ? exp(l64 - (double)mx) / sum64 : 1.0 / (1.0 + exp(-l64));
        return order_key(s64 + (a.bias ? (double)a.bias[e] : 0.0));
    };
    // Adds to the n experts in cand those of this lane whose key is at least `floor`
    // (0: none); returns their number, which may be above 32.
    auto collect = [&](int n, uint32_t floor) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const bool c = floor != 0u && key[i] >= floor;
            const unsigned mask = __ballot_sync(0xffffffffu, c);
            const int at = n + __popc(mask & ((1u << lane) - 1u));
            if (c && at < 32)
                cand[at] = grp * a.gs + sub + a.lg * i;
            n += __popc(mask);
        }
        __syncwarp();
        return n;
    };

    bool sure = true;
    if (a.k_groups < a.n_groups) {
        for (int o = 1; o < a.lg; o <<= 1) {
            const uint32_t o1 = __shfl_xor_sync(0xffffffffu, b1, o), o2 = __shfl_xor_sync(0xffffffffu, b2, o);
            b2 = max(max(b2, o2), min(b1, o1));
            b1 = max(b1, o1);
        }
        uint32_t gk = b1;
        if (a.top2 && b2 != 0u)
            gk = order_key32(key_value32(b1) + key_value32(b2));
        // rank of the group's score among all (groups with every expert off rank last)
        bool kept = false;
        uint32_t last = 0u;
        for (int r = 0; r <= a.k_groups; ++r) {
            const uint32_t v = has_grp && !kept ? gk : 0u;
            const uint32_t m = __reduce_max_sync(0xffffffffu, v);
            if (r == a.k_groups) {
                // the gap between the last group that stays and the next (sums of two keys, rounded)
                if (m != 0u) {
                    const float x = key_value32(last), y = key_value32(m);
                    const float tol = 1.01f * (2.f * err_of(x) + 4.f * U * (fabsf(x) + fabsf(y)));
                    if (x - y <= tol) {
                        // Groups above y + tol stay and groups below x - tol do not; the FP64
                        // scores of those between decide.  A score is that of the experts whose
                        // keys can be the largest, or the second largest, of the group.
                        const float g = key_value32(gk);
                        const bool in = has_grp && gk != 0u && g > y + tol;
                        const bool open = has_grp && gk != 0u && !in && g >= x - tol;
                        const int left = a.k_groups - __popc(__ballot_sync(0xffffffffu, in && sub == 0));
                        const uint32_t low = a.top2 ? b2 : b1;
                        const uint32_t floor =
                            low == 0u ? 1u : order_key32(key_value32(low) - err_of(key_value32(b1)));
                        const int n = collect(0, open ? floor : 0u);
                        if (n > 32)
                            return false;
                        const int e = lane < n ? cand[lane] : 0, eg = lane < n ? e / a.gs : -1;
                        const u64 k64 = keys64(e, lane < n);
                        u64 g1 = 0ull, g2 = 0ull;
                        bool repeats = false;  // an earlier lane stands for the group
                        for (int j = 0; j < n; ++j) {
                            const u64 kj = __shfl_sync(0xffffffffu, k64, j);
                            if (__shfl_sync(0xffffffffu, eg, j) == eg) {
                                g2 = max(g2, min(g1, kj));
                                g1 = max(g1, kj);
                                repeats = repeats || j < lane;
                            }
                        }
                        const u64 g64 = a.top2 && g2 != 0ull ? order_key(key_value(g1) + key_value(g2)) : g1;
                        int better = 0;
                        for (int j = 0; j < n; ++j) {
                            const u64 gj = __shfl_sync(0xffffffffu, g64, j);
                            const int ej = __shfl_sync(0xffffffffu, repeats ? -1 : eg, j);
                            better += ej >= 0 && (gj > g64 || (gj == g64 && ej < eg));
                        }
                        kept = in;
                        for (int j = 0; j < n; ++j) {
                            const int ej = __shfl_sync(0xffffffffu, better < left ? eg : -1, j);
                            kept = kept || ej == grp;
                        }
                        __syncwarp();  // cand is written again
                    }
                }
                break;
            }
            if (m == 0u)
                break;  // the groups left have every expert off
            const int src = __ffs(__ballot_sync(0xffffffffu, v == m)) - 1;
            kept = kept || grp == src / a.lg;
            last = m;
        }
        if (!kept)
#pragma unroll
            for (int i = 0; i < NV; ++i)
                key[i] = 0u;
    }

    int my_e = -1, taken = 0;
    uint32_t prev = 0u;
    for (int j = 0; j <= a.k; ++j) {
        uint32_t best = key[0];
#pragma unroll
        for (int i = 1; i < NV; ++i)
            best = max(best, key[i]);
        const uint32_t m = __reduce_max_sync(0xffffffffu, best);
        if (m == 0u)
            break;  // no expert is left: empty slots
        if (j > 0) {
            const float x = key_value32(prev), gap = x - key_value32(m);
            // (a gap that any softmax score's error allows for needs no logarithm)
            if (SCORE != MOE_SCORE_SOFTMAX || a.bias || !(gap > 1024.f * U * x))
                sure = sure && gap > err_of(x);
        }
        if (j == a.k)
            break;
        prev = m;
        const int src = __ffs(__ballot_sync(0xffffffffu, best == m)) - 1;
        int e = 0;
        bool hit = lane != src;  // take one key of that lane (an equal one stays and leaves no gap)
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (!hit && key[i] == m) {
                hit = true;
                e = i;
                key[i] = 0u;
            }
        e = __shfl_sync(0xffffffffu, grp * a.gs + sub + a.lg * e, src);
        if (lane == j)
            my_e = e;
        taken = j + 1;
    }
    if (!sure) {
        // Candidates: the experts taken, and the others whose key can reach the last
        // taken one's (within twice the error).
        const float last = key_value32(prev);
        const uint32_t floor_key = order_key32(last - err_of(last));
        if (lane < taken)
            cand[lane] = my_e;
        const int n = collect(taken, floor_key);
        if (n > 32)
            return false;
        const int e = lane < n ? cand[lane] : 0;
        const u64 k64 = keys64(e, lane < n);
        int rank = 0;
        for (int j = 0; j < n; ++j) {
            const u64 kj = __shfl_sync(0xffffffffu, k64, j);
            const int ej = __shfl_sync(0xffffffffu, e, j);
            rank += kj > k64 || (kj == k64 && ej < e);
        }
        __syncwarp();
        if (lane < n && rank < taken)
            cand[rank] = e;
        __syncwarp();
        my_e = lane < taken ? cand[lane] : -1;
    }
    float s = 0.f;
    if (my_e >= 0)
        s = SCORE == MOE_SCORE_SOFTMAX ? expf(row[my_e] - mx) / inv : 1.f / (1.f + expf(-row[my_e]));
    if (a.renorm) {
        float tot = s;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            tot += __shfl_xor_sync(0xffffffffu, tot, o);
        s = tot == 0.f ? 0.f : s / tot;
    }
    if (lane < a.k) {
        a.ids[t * a.k + lane] = my_e;
        a.w[t * a.k + lane] = my_e >= 0 ? a.scale * s : 0.f;
    }
    return true;
}

template <int SCORE, int NV>
__global__ void __launch_bounds__(ROUTE_THREADS) route_grouped_kernel(const __grid_constant__ RouteArgs a)
{
    __shared__ int cand[ROUTE_THREADS / 32][32];
    overlap_trigger();
    overlap_wait();
    const long long t = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    if (t < a.T && !route_fast<SCORE, NV>(a, t, cand[threadIdx.x >> 5]))
        route_exact<SCORE, NV>(a, t);
}

template <int SCORE>
cudaError_t launch(const RouteArgs &a, cudaStream_t st)
{
    constexpr int threads = ROUTE_THREADS;
    const unsigned blocks = (unsigned)(((long long)a.T * 32 + threads - 1) / threads);
    const int nv = (a.gs + a.lg - 1) / a.lg;
#define MOE_GROUPED_CASE(N)                                          \
    if (nv <= N)                                                     \
        return launch_overlapped(route_grouped_kernel<SCORE, N>, blocks, threads, 0, 1, st, a);
    MOE_GROUPED_CASE(4)
    MOE_GROUPED_CASE(8)
    MOE_GROUPED_CASE(16)
    MOE_GROUPED_CASE(32)
    MOE_GROUPED_CASE(64)
#undef MOE_GROUPED_CASE
    return cudaErrorInvalidValue;
}

MoeStatus bad(MoeStatus s, const char *msg) { return (MoeStatus)set_last_error(s, msg); }

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" MoeStatus moe_route_grouped(const float *router_logits, const float *bias, int T, int E, int k,
                                       int n_groups, int k_groups, MoeScore score, MoeGroupScore group_score,
                                       int renormalize, float scale, int32_t *topk_ids, float *topk_w,
                                       void *cuda_stream)
{
    char msg[160];
    if (T < 0 || T > (1 << 24)) {
        snprintf(msg, sizeof msg, "T = %d out of range [0, 2^24]", T);
        return bad(MOE_EINVAL, msg);
    }
    if (E < 1 || E > MOE_ROUTE_GROUPED_MAX_EXPERTS) {
        snprintf(msg, sizeof msg, "E = %d out of range [1, %d]", E, MOE_ROUTE_GROUPED_MAX_EXPERTS);
        return bad(MOE_EINVAL, msg);
    }
    if (n_groups < 1 || n_groups > MOE_ROUTE_GROUPED_MAX_GROUPS || E % n_groups) {
        snprintf(msg, sizeof msg, "n_groups = %d must divide E = %d and lie in [1, %d]", n_groups, E,
                 MOE_ROUTE_GROUPED_MAX_GROUPS);
        return bad(MOE_EINVAL, msg);
    }
    if (k_groups < 1 || k_groups > n_groups) {
        snprintf(msg, sizeof msg, "k_groups = %d out of range [1, %d]", k_groups, n_groups);
        return bad(MOE_EINVAL, msg);
    }
    const int most = k_groups * (E / n_groups) < 32 ? k_groups * (E / n_groups) : 32;
    if (k < 1 || k > most) {
        snprintf(msg, sizeof msg, "k = %d out of range [1, min(32, k_groups * E / n_groups)] = [1, %d]", k, most);
        return bad(MOE_EINVAL, msg);
    }
    if ((score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) ||
        (group_score != MOE_GROUP_MAX && group_score != MOE_GROUP_TOP2))
        return bad(MOE_EINVAL, "moe_route_grouped: unknown score or group score");
    if (T == 0)
        return MOE_OK;
    if (!router_logits || !topk_ids || !topk_w)
        return bad(MOE_EINVAL, "moe_route_grouped: NULL pointer");
    if (((uintptr_t)router_logits | (uintptr_t)bias | (uintptr_t)topk_ids | (uintptr_t)topk_w) % 4)
        return bad(MOE_EINVAL, "moe_route_grouped: arrays must be 4-byte aligned");
    RouteArgs a{};
    a.logits = router_logits;
    a.bias = bias;
    a.T = T;
    a.E = E;
    a.k = k;
    a.n_groups = n_groups;
    a.k_groups = k_groups;
    a.gs = E / n_groups;
    a.lg = 32;
    while (a.lg * n_groups > 32)
        a.lg >>= 1;
    a.top2 = group_score == MOE_GROUP_TOP2;
    a.renorm = renormalize != 0;
    a.scale = scale;
    a.ids = topk_ids;
    a.w = topk_w;
    const cudaError_t e = score == MOE_SCORE_SOFTMAX ? launch<MOE_SCORE_SOFTMAX>(a, (cudaStream_t)cuda_stream)
                                                     : launch<MOE_SCORE_SIGMOID>(a, (cudaStream_t)cuda_stream);
    if (e != cudaSuccess) {
        snprintf(msg, sizeof msg, "grouped router launch: %s", cudaGetErrorString(e));
        return bad(MOE_ECUDA, msg);
    }
    return MOE_OK;
}
