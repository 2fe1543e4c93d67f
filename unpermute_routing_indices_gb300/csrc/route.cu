// The router of current mixture models: softmax or sigmoid scores, a bias for
// balance, groups of experts, top-K, renormalised weights; and its gradient.
//
//   s_e = softmax(l)_e or sigmoid(l_e);  c_e = s_e + b_e decides the choice
//   weights: scale * s_k / sum_j s_j (renorm) or scale * s_k
//
// k_route: one warp per token; lane l holds the experts l, l+32, ...  The choice
// is made in 64 bits, where scores next to each other stay apart; the weights
// are fp32.
#include <cfloat>
#include <climits>
#include <cuda_fp16.h>

#include "common.cuh"

namespace mp {
namespace {

constexpr int RT_THREADS = 256;
constexpr int RT_WARPS = RT_THREADS / 32;

struct RouteArgs {
    const void *logits;
    const float *bias;
    int64_t T;
    int E, K, score, n_groups, topk_groups, group_top, renorm;
    float scale;
    int32_t *idx;
    float *weights;
};

__device__ __forceinline__ float logit(const float *p) { return __ldg(p); }
__device__ __forceinline__ float logit(const __nv_bfloat16 *p)
{
    return __uint_as_float(static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t *>(p))) << 16);
}
__device__ __forceinline__ float logit(const __half *p) { return __half2float(__ldg(p)); }

__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(__half *p, float v) { *p = __float2half_rn(v); }

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL_MASK, v, d));
    return v;
}
template <typename F> __device__ __forceinline__ F warp_sum(F v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(FULL_MASK, v, d);
    return v;
}

// Arg-max of (value desc, index asc) across the warp; index INT_MAX: no candidate.
__device__ __forceinline__ void warp_argmax(double &v, int &i)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        const double ov = __shfl_xor_sync(FULL_MASK, v, d);
        const int oi = __shfl_xor_sync(FULL_MASK, i, d);
        if (oi != INT_MAX && (i == INT_MAX || ov > v || (ov == v && oi < i))) {
            v = ov;
            i = oi;
        }
    }
}

// A logit that can be chosen: not -inf and not NaN (an unavailable expert);
// +inf counts as the largest finite value.
__device__ __forceinline__ bool usable(float v) { return v > -INFINITY; }

// The choice in 64 bits.  `live`: bit j for expert lane + 32 j.  Lane k gets
// pick k (-1: none left).
template <int PER>
__device__ __forceinline__ int choose_exact(const RouteArgs &a, const float (&v)[PER],
                                            const float (&b)[PER], unsigned have, unsigned live,
                                            int lane)
{
    double c[PER];
    if (a.score == MP_SCORE_SIGMOID) {
#pragma unroll
        for (int j = 0; j < PER; ++j) c[j] = 1.0 / (1.0 + exp(-static_cast<double>(v[j])));
    } else {
        float m = -INFINITY;
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if (have >> j & 1u) m = fmaxf(m, v[j]);
        m = warp_max(m);
        double s = 0.0;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            c[j] = (have >> j & 1u) ? exp(static_cast<double>(v[j]) - m) : 0.0;
            s += c[j];
        }
        s = warp_sum(s);
#pragma unroll
        for (int j = 0; j < PER; ++j) c[j] /= s;
    }
    if (a.bias != nullptr)
#pragma unroll
        for (int j = 0; j < PER; ++j) c[j] += static_cast<double>(b[j]);

    if (a.n_groups > 1) {
        const int per_group = a.E / a.n_groups;
        double worth = 0.0;          // lane g: group g's
        int mine = INT_MAX;          // lane g: g, if the group has an expert
        for (int g = 0; g < a.n_groups; ++g) {
            double total = 0.0;
            int first = INT_MAX;
            for (int r = 0; r < a.group_top; ++r) {
                double bv = 0.0;
                int bi = INT_MAX;
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    const int e = lane + 32 * j;
                    if ((live >> j & 1u) && e / per_group == g && e != first &&
                        (bi == INT_MAX || c[j] > bv)) {
                        bv = c[j];
                        bi = e;
                    }
                }
                warp_argmax(bv, bi);
                if (bi != INT_MAX) total += bv;
                if (r == 0) first = bi;
            }
            if (lane == g) {
                worth = total;
                mine = first == INT_MAX ? INT_MAX : g;
            }
        }
        unsigned kept = 0;
        for (int r = 0; r < a.topk_groups; ++r) {
            double bv = worth;
            int bi = (mine != INT_MAX && !(kept >> lane & 1u)) ? mine : INT_MAX;
            warp_argmax(bv, bi);
            if (bi != INT_MAX) kept |= 1u << bi;
        }
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if ((live >> j & 1u) && !(kept >> ((lane + 32 * j) / per_group) & 1u)) live &= ~(1u << j);
    }
    // Without a bias the scores rise with the logits, which stay apart where
    // scores round to one value.
    if (a.bias == nullptr)
#pragma unroll
        for (int j = 0; j < PER; ++j) c[j] = static_cast<double>(v[j]);
    int pick = -1;
    for (int k = 0; k < a.K; ++k) {
        double bv = 0.0;
        int bi = INT_MAX;
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if ((live >> j & 1u) && (bi == INT_MAX || c[j] > bv)) {
                bv = c[j];
                bi = lane + 32 * j;
            }
        warp_argmax(bv, bi);
        if (bi == INT_MAX) break;
        if ((bi & 31) == lane) live &= ~(1u << (bi >> 5));
        if (lane == k) pick = bi;
    }
    return pick;
}

template <typename L, int PER>
__global__ void __launch_bounds__(RT_THREADS) k_route(const RouteArgs a)
{
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * RT_WARPS + (threadIdx.x >> 5);
    if (t >= a.T) return;   // whole warps leave together
    const L *l = static_cast<const L *>(a.logits) + t * a.E;
    float v[PER], b[PER];
    unsigned have = 0, live = 0;   // has a logit; can be chosen
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int e = lane + 32 * j;
        v[j] = e < a.E ? fminf(logit(l + e), FLT_MAX) : -INFINITY;
        b[j] = (e < a.E && a.bias != nullptr) ? __ldg(a.bias + e) : 0.0f;
        if (e < a.E && isnan(logit(l + e))) v[j] = -INFINITY;
        if (usable(v[j])) {
            have |= 1u << j;
            if (usable(b[j])) live |= 1u << j;
        }
    }
    const int pick = choose_exact<PER>(a, v, b, have, live, lane);

    // The weights.  sigmoid(v) is exp(v) for v far below zero; where all
    // picks are there, their ratio is taken from exp(v_k - m), which does not
    // underflow.
    const float pv = pick >= 0 ? fminf(logit(l + pick), FLT_MAX) : -INFINITY;
    const float m = warp_max(pv);
    float s;
    if (a.score == MP_SCORE_SIGMOID && !(a.renorm && m < -40.0f))
        s = pick >= 0 ? __fdiv_rn(1.0f, 1.0f + expf(-pv)) : 0.0f;
    else if (a.score == MP_SCORE_SIGMOID || a.renorm)
        s = pick >= 0 ? expf(pv - m) : 0.0f;
    else {
        float top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int j = 0; j < PER; ++j) top = fmaxf(top, v[j]);
        top = warp_max(top);
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if (have >> j & 1u) sum += expf(v[j] - top);
        sum = warp_sum(sum);
        s = pick >= 0 ? __fdiv_rn(expf(pv - top), sum) : 0.0f;
    }
    if (a.renorm) s = __fdiv_rn(s, warp_sum(s));
    if (lane < a.K) {
        a.idx[t * a.K + lane] = pick;
        a.weights[t * a.K + lane] = pick >= 0 ? a.scale * s : 0.0f;
    }
}

struct RouteBwdArgs {
    const float *g_weights;
    const void *logits;
    const int32_t *idx;
    int64_t T;
    int E, K, score, renorm;
    float scale;
    void *g_logits;
};

// renorm: with p the weights before scaling, g_l = scale p_k (g_k - sum_j g_j p_j),
// times 1 - s_k for the sigmoid.  Raw weights: sigmoid scale g_k s_k (1 - s_k);
// softmax scale s_e ([e picked] g_k - sum_j g_j s_j) for every expert.
template <typename L, int PER>
__global__ void __launch_bounds__(RT_THREADS) k_route_bwd(const RouteBwdArgs a)
{
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * RT_WARPS + (threadIdx.x >> 5);
    if (t >= a.T) return;
    const L *l = static_cast<const L *>(a.logits) + t * a.E;
    L *gl = static_cast<L *>(a.g_logits) + t * a.E;
    int pick = lane < a.K ? __ldg(a.idx + t * a.K + lane) : -1;
    if (pick >= a.E) pick = -1;
    const float g = pick >= 0 ? a.scale * __ldg(a.g_weights + t * a.K + lane) : 0.0f;
    const float pv = pick >= 0 ? fminf(logit(l + pick), FLT_MAX) : -INFINITY;
    const bool dense = a.score == MP_SCORE_SOFTMAX && !a.renorm;
    float at_pick;
    if (!dense) {
        for (int e = lane; e < a.E; e += 32) put(gl + e, 0.0f);
        float left = 1.0f, s;   // 1 - s of the sigmoid
        const float m = warp_max(pv);
        if (a.score == MP_SCORE_SIGMOID) {
            left = __fdiv_rn(1.0f, 1.0f + expf(pv));
            s = (a.renorm && m < -40.0f) ? expf(pv - m) : __fdiv_rn(1.0f, 1.0f + expf(-pv));
        } else {
            s = expf(pv - m);
        }
        if (pick < 0) s = 0.0f;
        if (a.renorm) {
            const float p = __fdiv_rn(s, warp_sum(s));
            const float d = warp_sum(pick >= 0 ? g * p : 0.0f);
            at_pick = p * (g - d) * left;
        } else {
            at_pick = g * s * left;
        }
        __syncwarp();   // the zeros above land first
    } else {
        float v[PER], top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int e = lane + 32 * j;
            v[j] = e < a.E ? fminf(logit(l + e), FLT_MAX) : -INFINITY;
            if (e < a.E && isnan(logit(l + e))) v[j] = -INFINITY;
            top = fmaxf(top, v[j]);
        }
        top = warp_max(top);
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            v[j] = usable(v[j]) ? expf(v[j] - top) : 0.0f;
            sum += v[j];
        }
        sum = warp_sum(sum);
        const float inv = sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
        const float s = pick >= 0 ? expf(pv - top) * inv : 0.0f;
        const float d = warp_sum(pick >= 0 ? g * s : 0.0f);
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int e = lane + 32 * j;
            if (e < a.E) put(gl + e, -v[j] * inv * d);
        }
        at_pick = s * (g - d);
        __syncwarp();
    }
    if (pick >= 0) put(gl + pick, at_pick);
}

template <typename L> mp_status_t launch_route(const RouteArgs &a, cudaStream_t s)
{
    const unsigned blocks = static_cast<unsigned>((a.T + RT_WARPS - 1) / RT_WARPS);
    const int per = (a.E + 31) / 32;
    if (per <= 4)
        (void)launch_pdl(k_route<L, 4>, blocks, RT_THREADS, 0, s, a);
    else if (per <= 8)
        (void)launch_pdl(k_route<L, 8>, blocks, RT_THREADS, 0, s, a);
    else if (per <= 16)
        (void)launch_pdl(k_route<L, 16>, blocks, RT_THREADS, 0, s, a);
    else
        (void)launch_pdl(k_route<L, 32>, blocks, RT_THREADS, 0, s, a);
    return check_launch();
}

template <typename L> mp_status_t launch_route_bwd(const RouteBwdArgs &a, cudaStream_t s)
{
    const unsigned blocks = static_cast<unsigned>((a.T + RT_WARPS - 1) / RT_WARPS);
    const int per = (a.E + 31) / 32;
    if (per <= 8)
        (void)launch_pdl(k_route_bwd<L, 8>, blocks, RT_THREADS, 0, s, a);
    else
        (void)launch_pdl(k_route_bwd<L, 32>, blocks, RT_THREADS, 0, s, a);
    return check_launch();
}

mp_status_t route_sizes(int64_t T, int32_t E, int32_t K, int32_t score, int32_t dtype)
{
    if (T < 0 || E < 1 || K < 1 || K > E || score < MP_SCORE_SOFTMAX || score > MP_SCORE_SIGMOID ||
        dtype < MP_DTYPE_BF16 || dtype > MP_DTYPE_FP32)
        return MP_ERR_INVALID_ARG;
    if (E > MP_MAX_EXPERTS || K > 32 || T > INT32_MAX) return MP_ERR_UNSUPPORTED;
    return MP_OK;
}

}  // namespace
}  // namespace mp

using namespace mp;

extern "C" mp_status_t mp_route(const void *logits, int32_t dtype, const float *bias, int64_t T,
                                int32_t E, int32_t K, int32_t score, int32_t n_groups,
                                int32_t topk_groups, int32_t group_top, int32_t renorm,
                                float scale, int32_t *idx, float *weights, mp_stream_t stream)
{
    if (const mp_status_t s = route_sizes(T, E, K, score, dtype); s != MP_OK) return s;
    if (n_groups < 1 || topk_groups < 1 || group_top < 1 || group_top > 2)
        return MP_ERR_INVALID_ARG;
    if (n_groups > 32) return MP_ERR_UNSUPPORTED;
    if (E % n_groups != 0 || topk_groups > n_groups ||
        static_cast<int64_t>(topk_groups) * (E / n_groups) < K)
        return MP_ERR_INVALID_ARG;
    if (T == 0) return MP_OK;
    if (logits == nullptr || idx == nullptr || weights == nullptr) return MP_ERR_INVALID_ARG;
    const RouteArgs a = {logits, bias, T, E, K, score, n_groups, topk_groups, group_top, renorm,
                         scale, idx, weights};
    const cudaStream_t s = as_stream(stream);
    return dtype == MP_DTYPE_FP32   ? launch_route<float>(a, s)
           : dtype == MP_DTYPE_BF16 ? launch_route<__nv_bfloat16>(a, s)
                                    : launch_route<__half>(a, s);
}

extern "C" mp_status_t mp_route_bwd(const float *g_weights, const void *logits, int32_t dtype,
                                    const int32_t *idx, int64_t T, int32_t E, int32_t K,
                                    int32_t score, int32_t renorm, float scale, void *g_logits,
                                    mp_stream_t stream)
{
    if (const mp_status_t s = route_sizes(T, E, K, score, dtype); s != MP_OK) return s;
    if (T == 0) return MP_OK;
    if (g_weights == nullptr || logits == nullptr || idx == nullptr || g_logits == nullptr)
        return MP_ERR_INVALID_ARG;
    const RouteBwdArgs a = {g_weights, logits, idx, T, E, K, score, renorm, scale, g_logits};
    const cudaStream_t s = as_stream(stream);
    return dtype == MP_DTYPE_FP32   ? launch_route_bwd<float>(a, s)
           : dtype == MP_DTYPE_BF16 ? launch_route_bwd<__nv_bfloat16>(a, s)
                                    : launch_route_bwd<__half>(a, s);
}
