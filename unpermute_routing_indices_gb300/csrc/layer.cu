// The whole mixture-of-experts layer for a few tokens.
//
//   l = x router^T;  (idx, w) = the router's choice;
//   y[t] = sum_k w[t,k] (act(x[t] w1[e]^T + b1[e]) w2[e]^T + b2[e]),  e = idx[t,k]
//
// The logits are sums in pairs of fp32 (a sum and what its roundings lost), so that
// they are those of 64 bits rounded once, and the choice with them.
#include "expert.cuh"
#include "route.cuh"
#include "tc.cuh"

namespace mp {
namespace {

constexpr int LAYER_THREADS = 256, LAYER_WARPS = LAYER_THREADS / 32;

struct LayerArgs {
    const mp_bf16_t *x, *w1, *b1, *w2, *b2;
    const void *router;
    RouteArgs route;
    int T, E, K, H, F, O, act;
    int32_t *idx;
    float *weights;
    mp_bf16_t *h, *y;
};

__device__ __forceinline__ float bf16_value(const mp_bf16_t *p)
{
    return __uint_as_float(static_cast<uint32_t>(__ldg(p)) << 16);
}

// A sum of fp32 values and what its roundings lost (Knuth's two-sum).
struct PairSum {
    float s = 0.0f, lost = 0.0f;
    __device__ __forceinline__ void add(float p)
    {
        const float t = __fadd_rn(s, p), z = __fsub_rn(t, s);
        lost = __fadd_rn(lost, __fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(p, z)));
        s = t;
    }
    // a b, and what the product's rounding lost (nothing for two bf16 values)
    template <bool EXACT> __device__ __forceinline__ void add_product(float a, float b)
    {
        const float p = __fmul_rn(a, b);
        if (!EXACT) lost = __fadd_rn(lost, __fmaf_rn(a, b, -p));
        add(p);
    }
    __device__ __forceinline__ float sum() const { return isfinite(s) ? __fadd_rn(s, lost) : s; }
};

template <typename L, int PER> __global__ void __launch_bounds__(LAYER_THREADS) k_layer_route(const LayerArgs a)
{
    extern __shared__ SharedLogit logits[];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = blockIdx.x;
    const mp_bf16_t *x = a.x + static_cast<int64_t>(t) * a.H;
    for (int e = warp; e < a.E; e += LAYER_WARPS) {
        const L *r = static_cast<const L *>(a.router) + static_cast<int64_t>(e) * a.H;
        PairSum v;
        for (int c = lane; c < a.H; c += 32) v.add_product<sizeof(L) == 2>(bf16_value(x + c), logit(r + c));
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            const float s = __shfl_xor_sync(FULL_MASK, v.s, d), lost = __shfl_xor_sync(FULL_MASK, v.lost, d);
            v.add(s);
            v.lost = __fadd_rn(v.lost, lost);
        }
        if (lane == 0) logits[e].v = v.sum();
    }
    __syncthreads();
    if (warp == 0) route_token<SharedLogit, PER, 0>(a.route, logits, t, lane);
}

__device__ __forceinline__ float act_of(int act, float z)
{
    switch (act_inner(act)) {
    case MP_ACT_SILU: return act_value<MP_ACT_SILU>(z);
    case MP_ACT_GELU: return act_value<MP_ACT_GELU>(z);
    case MP_ACT_RELU: return act_value<MP_ACT_RELU>(z);
    default: return z;
    }
}

__device__ __forceinline__ float warp_dot(const mp_bf16_t *a, const mp_bf16_t *b, int n, int lane)
{
    float v = 0.0f;
    for (int c = lane; c < n; c += 32) v = fmaf(bf16_value(a + c), bf16_value(b + c), v);
    return warp_sum(v);
}

// h[t,k,f]: a warp each.
__global__ void __launch_bounds__(LAYER_THREADS) k_layer_up(const LayerArgs a)
{
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, f = blockIdx.x * LAYER_WARPS + (threadIdx.x >> 5), r = blockIdx.y;
    const int e = a.idx[r];
    if (f >= a.F || e < 0) return;
    const bool gated = act_gated(a.act);
    const int64_t P = static_cast<int64_t>(a.F) * (gated ? 2 : 1);
    const mp_bf16_t *x = a.x + static_cast<int64_t>(r / a.K) * a.H;
    float z = warp_dot(x, a.w1 + (e * P + f) * a.H, a.H, lane);
    if (a.b1 != nullptr) z += bf16_value(a.b1 + e * P + f);
    z = act_of(a.act, z);
    if (gated) {
        float u = warp_dot(x, a.w1 + (e * P + a.F + f) * a.H, a.H, lane);
        if (a.b1 != nullptr) u += bf16_value(a.b1 + e * P + a.F + f);
        z *= u;
    }
    const float v[1] = {z};
    if (lane == 0) a.h[static_cast<int64_t>(r) * a.F + f] = pack(v);
}

// y[t,o]: a warp each, the experts in the order of their slots.
__global__ void __launch_bounds__(LAYER_THREADS) k_layer_down(const LayerArgs a)
{
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, o = blockIdx.x * LAYER_WARPS + (threadIdx.x >> 5), t = blockIdx.y;
    if (o >= a.O) return;
    float y = 0.0f;
    for (int k = 0; k < a.K; ++k) {
        const int64_t r = static_cast<int64_t>(t) * a.K + k;
        const int e = a.idx[r];
        if (e < 0) continue;
        const int64_t row = static_cast<int64_t>(e) * a.O + o;
        float v = 0.0f;   // h is of the kernel before: no loads past the coherent path
        for (int c = lane; c < a.F; c += 32) {
            float h[1];
            unpack(a.h[r * a.F + c], h);
            v = fmaf(h[0], bf16_value(a.w2 + row * a.F + c), v);
        }
        v = warp_sum(v);
        if (a.b2 != nullptr) v += bf16_value(a.b2 + row);
        y = fmaf(a.weights[r], v, y);
    }
    const float v[1] = {y};
    if (lane == 0) a.y[static_cast<int64_t>(t) * a.O + o] = pack(v);
}

template <typename L> void launch_layer_route(const LayerArgs &a, cudaStream_t s)
{
    const size_t smem = a.E * sizeof(SharedLogit);
    if (a.E <= 128)
        (void)launch_pdl(k_layer_route<L, 4>, a.T, LAYER_THREADS, smem, s, a);
    else if (a.E <= 256)
        (void)launch_pdl(k_layer_route<L, 8>, a.T, LAYER_THREADS, smem, s, a);
    else
        (void)launch_pdl(k_layer_route<L, 32>, a.T, LAYER_THREADS, smem, s, a);
}

mp_status_t layer_sizes(int64_t T, int32_t E, int32_t K, int32_t H, int32_t F, int32_t O)
{
    if (T < 0 || E < 1 || K < 1 || K > E || H < 1 || F < 1 || O < 1) return MP_ERR_INVALID_ARG;
    constexpr int WIDEST = MP_MAX_LAYER_WIDTH;
    return T > MP_MAX_LAYER_TOKENS || E > MP_MAX_EXPERTS || K > 32 || H > WIDEST || F > WIDEST || O > WIDEST
               ? MP_ERR_UNSUPPORTED
               : MP_OK;
}

}  // namespace
}  // namespace mp

using namespace mp;

extern "C" size_t mp_moe_layer_workspace_size(int64_t T, int32_t E, int32_t K, int32_t H, int32_t F, int32_t O)
{
    if (layer_sizes(T, E, K, H, F, O) != MP_OK) return 0;
    const size_t bytes = static_cast<size_t>(T) * K * F * sizeof(mp_bf16_t);
    return bytes < 256 ? 256 : (bytes + 255) / 256 * 256;
}

extern "C" mp_status_t mp_moe_layer(const mp_bf16_t *x, const void *router, int32_t router_dtype,
                                    const float *bias, const mp_bf16_t *w1, const mp_bf16_t *b1,
                                    const mp_bf16_t *w2, const mp_bf16_t *b2, int64_t T, int32_t E, int32_t K,
                                    int32_t H, int32_t F, int32_t O, int32_t act, int32_t score, int32_t n_groups,
                                    int32_t topk_groups, int32_t group_top, int32_t renorm, float scale,
                                    int32_t *idx, float *weights, mp_bf16_t *y, void *workspace,
                                    size_t workspace_bytes, int32_t *dev_status, mp_stream_t stream)
{
    if (const mp_status_t s = layer_sizes(T, E, K, H, F, O); s != MP_OK) return s;
    if (const mp_status_t s = route_sizes(T, E, K, score, router_dtype); s != MP_OK) return s;
    if (act < MP_ACT_NONE || act > MP_ACT_SWIGLU) return MP_ERR_INVALID_ARG;
    RouteArgs route;
    if (const mp_status_t s = route_args(route, bias, E, K, score, n_groups, topk_groups, group_top, renorm, scale);
        s != MP_OK)
        return s;
    if (T == 0) return MP_OK;
    if (x == nullptr || router == nullptr || w1 == nullptr || w2 == nullptr || idx == nullptr ||
        weights == nullptr || y == nullptr)
        return MP_ERR_INVALID_ARG;
    if (workspace == nullptr || !aligned16(workspace) ||
        workspace_bytes < mp_moe_layer_workspace_size(T, E, K, H, F, O))
        return MP_ERR_WORKSPACE;
    (void)dev_status;
    route.T = T; route.idx = idx; route.weights = weights;
    const cudaStream_t s = as_stream(stream);
    const LayerArgs a = {x, w1, b1, w2, b2, router, route, static_cast<int>(T), E, K, H, F, O, act, idx, weights,
                         static_cast<mp_bf16_t *>(workspace), y};
    switch (router_dtype) {
    case MP_DTYPE_BF16: launch_layer_route<__nv_bfloat16>(a, s); break;
    case MP_DTYPE_FP16: launch_layer_route<__half>(a, s); break;
    default: launch_layer_route<float>(a, s); break;
    }
    const unsigned rows = static_cast<unsigned>(T * K);
    (void)launch_pdl(k_layer_up, dim3((F + LAYER_WARPS - 1) / LAYER_WARPS, rows), LAYER_THREADS, 0, s, a);
    (void)launch_pdl(k_layer_down, dim3((O + LAYER_WARPS - 1) / LAYER_WARPS, static_cast<unsigned>(T)),
                     LAYER_THREADS, 0, s, a);
    return check_launch();
}
