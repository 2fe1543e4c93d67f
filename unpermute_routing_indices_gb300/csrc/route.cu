// The router of current mixture models: softmax or sigmoid scores, a bias for
// balance, groups of experts, top-K, renormalised weights; and its gradient.
//
//   s_e = softmax(l)_e or sigmoid(l_e);  c_e = s_e + b_e decides the choice
//   weights: scale * s_k / sum_j s_j (renorm) or scale * s_k
//
// k_route: one warp per token; lane l holds the experts l, l+32, ...
// Choice.  Without a bias the scores rise with the logits, which are compared
// as they are.  With one, and for the sum of a group's best two, fp32 values of
// c decide wherever neighbours in the order are further apart than their errors
// can be (too_near); a token where two are nearer (about one of two thousand of
// normal logits) is decided again in 64 bits: the two groups or the picks and the best
// of the rest where that is enough, else everything (choose_exact).  So the choice is
// that of 64 bits everywhere, at the cost of 32: on 32,768 tokens of 256 experts
// (sigmoid, bias, 8 groups), all of it in 64 bits took 1,290 us, this 39 (43 with choose_exact for all near tokens).
// Each lane sorts its candidates by a fixed network and a round takes the best
// head of the warp (topk.cuh); the round after the K-th says how near the best
// of the rest is.
// Weights are fp32 from the picks' own logits.
// k_route_bwd: one warp per token; every gradient is written once.
#include "route.cuh"

namespace mp {
namespace {

constexpr int RT_THREADS = 256;
constexpr int RT_WARPS = RT_THREADS / 32;

// KT > 0: a form for K = KT with the rounds unrolled (K = 8, kernels alone: 32,768 x 256,
// sigmoid, bias 32.6 -> 29.7 us, with groups 41.5 -> 40.3, softmax without a bias 29.1 -> 26.2;
// 16,384 x 128 11.3 -> 10.4, raw bf16 11.7 -> 11.3).  Compiled for 4 CTAs per
// SM up to 256 experts (32,768 x 256, sigmoid, bias: 41.4 us with 3, 38.7 with 4
// when this was chosen, 28.7 now), 3 up to 512 (16,383 x 512: 64.5 us with 1, 51.9 with 2,
// 48.7 with 3; 29 now) and 2 up to 1,024 (106.8 with 1, 90.9 with 2; 60 now).
template <typename L, int PER, int KT>
__global__ void __launch_bounds__(RT_THREADS, PER <= 8 ? 4 : PER <= 16 ? 3 : 2) k_route(const RouteArgs a)
{
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * RT_WARPS + (threadIdx.x >> 5);
    if (t >= a.T) return;   // whole warps leave together
    const L *l = static_cast<const L *>(a.logits) + t * a.E;
    route_token<L, PER, KT>(a, l, t, lane);
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
// VEC: the row is whole chunks of 4 logits, aligned: lane l then holds chunks l,
// l+32, ...; otherwise single ones.
template <typename L, int W> struct alignas(sizeof(L) * W) Chunk {
    L at[W];
};

template <typename L, int PER, bool VEC>
__global__ void __launch_bounds__(RT_THREADS) k_route_bwd(const RouteBwdArgs a)
{
    pdl_trigger();
    pdl_wait();
    constexpr int W = VEC ? 4 : 1, CHUNKS = PER / W;
    typedef Chunk<L, W> C;
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * RT_WARPS + (threadIdx.x >> 5);
    if (t >= a.T) return;
    const L *l = static_cast<const L *>(a.logits) + t * a.E;
    L *gl = static_cast<L *>(a.g_logits) + t * a.E;
    int pick = lane < a.K ? ld_in(a.idx + t * a.K + lane) : -1;
    if (pick >= a.E) pick = -1;
    const float g = pick >= 0 ? a.scale * ld_in(a.g_weights + t * a.K + lane) : 0.0f;
    const float pv = pick >= 0 ? fminf(logit(l + pick), FLT_MAX) : -INFINITY;
    const bool dense = a.score == MP_SCORE_SOFTMAX && !a.renorm;
    float at_pick;
    if (!dense) {
        C zero;
#pragma unroll
        for (int i = 0; i < W; ++i) put(zero.at + i, 0.0f);
        for (int e = lane * W; e < a.E; e += 32 * W) *reinterpret_cast<C *>(gl + e) = zero;
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
    } else {
        float v[CHUNKS][W], top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int j = 0; j < CHUNKS; ++j) {
            const int e = (lane + 32 * j) * W;
            C x;
            if (e < a.E) x = *reinterpret_cast<const C *>(l + e);
#pragma unroll
            for (int i = 0; i < W; ++i) {
                v[j][i] = e < a.E ? logit_value(x.at[i]) : -INFINITY;
                v[j][i] = usable(v[j][i]) ? fminf(v[j][i], FLT_MAX) : -INFINITY;
                top = fmaxf(top, v[j][i]);
            }
        }
        top = warp_max(top);
#pragma unroll
        for (int j = 0; j < CHUNKS; ++j)
#pragma unroll
            for (int i = 0; i < W; ++i) {
                v[j][i] = usable(v[j][i]) ? expf(v[j][i] - top) : 0.0f;
                sum += v[j][i];
            }
        sum = warp_sum(sum);
        const float inv = sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
        const float s = pick >= 0 ? expf(pv - top) * inv : 0.0f;
        const float d = warp_sum(pick >= 0 ? g * s : 0.0f);
#pragma unroll
        for (int j = 0; j < CHUNKS; ++j) {
            const int e = (lane + 32 * j) * W;
            C x;
#pragma unroll
            for (int i = 0; i < W; ++i) put(x.at + i, -v[j][i] * inv * d);
            if (e < a.E) *reinterpret_cast<C *>(gl + e) = x;
        }
        at_pick = s * (g - d);
    }
    __syncwarp();   // what is stored above lands before the picks' gradients
    if (pick >= 0) put(gl + pick, at_pick);
}

template <typename L> mp_status_t launch_route(const RouteArgs &a, cudaStream_t s)
{
    const unsigned blocks = static_cast<unsigned>((a.T + RT_WARPS - 1) / RT_WARPS);
    const int per = (a.E + 31) / 32;
    if (per <= 4 && a.K == 8)
        (void)launch_pdl(k_route<L, 4, 8>, blocks, RT_THREADS, 0, s, a);
    else if (per <= 8 && a.K == 8)
        (void)launch_pdl(k_route<L, 8, 8>, blocks, RT_THREADS, 0, s, a);
    else if (per <= 4)
        (void)launch_pdl(k_route<L, 4, 0>, blocks, RT_THREADS, 0, s, a);
    else if (per <= 8)
        (void)launch_pdl(k_route<L, 8, 0>, blocks, RT_THREADS, 0, s, a);
    else if (per <= 16)
        (void)launch_pdl(k_route<L, 16, 0>, blocks, RT_THREADS, 0, s, a);
    else
        (void)launch_pdl(k_route<L, 32, 0>, blocks, RT_THREADS, 0, s, a);
    return check_launch();
}

template <typename L> mp_status_t launch_route_bwd(const RouteBwdArgs &a, cudaStream_t s)
{
    const unsigned blocks = static_cast<unsigned>((a.T + RT_WARPS - 1) / RT_WARPS);
    const int per = (a.E + 31) / 32;
    const uintptr_t both = reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.g_logits);
    const bool vec = a.E % 4 == 0 && both % (4 * sizeof(L)) == 0;
    if (per <= 8 && vec)
        (void)launch_pdl(k_route_bwd<L, 8, true>, blocks, RT_THREADS, 0, s, a);
    else if (per <= 8)
        (void)launch_pdl(k_route_bwd<L, 8, false>, blocks, RT_THREADS, 0, s, a);
    else
        (void)launch_pdl(k_route_bwd<L, 32, false>, blocks, RT_THREADS, 0, s, a);
    return check_launch();
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
    RouteArgs a;
    if (const mp_status_t s = route_args(a, bias, E, K, score, n_groups, topk_groups, group_top, renorm, scale);
        s != MP_OK)
        return s;
    if (T == 0) return MP_OK;
    if (logits == nullptr || idx == nullptr || weights == nullptr) return MP_ERR_INVALID_ARG;
    a.logits = logits; a.T = T; a.idx = idx; a.weights = weights;
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
