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
#include <math.h>
#include <stdio.h>

#include "../../include/moe.h"
#include "moe_internal.cuh"

namespace moe {

namespace {

typedef unsigned long long u64;

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

template <int SCORE, int NV>
__global__ void route_grouped_kernel(const RouteArgs a)
{
    const int lane = threadIdx.x & 31;
    const long long t = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    if (t >= a.T)
        return;
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

template <int SCORE>
cudaError_t launch(const RouteArgs &a, cudaStream_t st)
{
    const int threads = 256;
    const unsigned blocks = (unsigned)(((long long)a.T * 32 + threads - 1) / threads);
    const int nv = (a.gs + a.lg - 1) / a.lg;
#define MOE_GROUPED_CASE(N)                                          \
    if (nv <= N) {                                                   \
        route_grouped_kernel<SCORE, N><<<blocks, threads, 0, st>>>(a); \
        return cudaGetLastError();                                   \
    }
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
