// The norms before and after a block, fused with the block's gate, residual scale
// and residual; and their gradients.
//
//   u = norm(x) w_post + b_post, or x;  s = residual + scale gate u
//   y = norm(s) w_pre + b_pre
//
// One CTA a row, the row in fp32 in shared memory.  The gradients of what is
// shared by the rows (weights, biases, a gate a channel) are summed in fp32 by each CTA over
// its rows, then over the CTAs in their order.
#include <cuda_fp16.h>

#include "common.cuh"

namespace mp {
namespace {

constexpr int NORM_THREADS = 256;
constexpr int NORM_PARTS = 152;   // partial sums of a shared gradient: a CTA an SM
constexpr int NORM_SHARED = 5;    // shared gradients at most: two weights, two biases, the gate

__device__ __forceinline__ float value(float v) { return v; }
__device__ __forceinline__ float value(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float value(__half v) { return __half2float(v); }
__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(__half *p, float v) { *p = __float2half_rn(v); }

template <typename D> struct NormArgs {
    const D *x, *residual, *post_w, *post_b, *gate, *pre_w, *pre_b;
    int64_t T;
    int H, kind, gate_form;
    float eps, scale;
    D *s, *y;
    float *stats;
};

// The sum over the CTA, in a fixed order.
__device__ __forceinline__ float cta_sum(float v, float *part)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(FULL_MASK, v, d);
    __syncthreads();   // what the last call left has been read
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.0f;
    for (int i = 0; i < NORM_THREADS / 32; ++i) t += part[i];
    return t;
}

template <typename D>
__device__ __forceinline__ float gate_at(const D *gate, int form, int64_t t, int c, int H)
{
    switch (form) {
    case MP_GATE_CHANNEL: return value(gate[c]);
    case MP_GATE_TOKEN: return value(gate[t]);
    case MP_GATE_ELEMENT: return value(gate[t * H + c]);
    default: return 1.0f;
    }
}

// Mean (0 for rms) and 1 / deviation of a row.  The deviations are taken from the mean,
// not from a difference of squares.
__device__ __forceinline__ void moments(const float *row, int H, int kind, float eps, float *part, float &mean,
                                        float &rstd)
{
    mean = 0.0f;
    if (kind == MP_NORM_LAYER) {
        float m = 0.0f;
        for (int c = threadIdx.x; c < H; c += NORM_THREADS) m += row[c];
        mean = cta_sum(m, part) / static_cast<float>(H);
    }
    float v = 0.0f;
    for (int c = threadIdx.x; c < H; c += NORM_THREADS) v += (row[c] - mean) * (row[c] - mean);
    rstd = 1.0f / sqrtf(cta_sum(v, part) / static_cast<float>(H) + eps);
}

template <typename D> __global__ void __launch_bounds__(NORM_THREADS) k_block_norm(const NormArgs<D> a)
{
    extern __shared__ float row[];
    __shared__ float part[NORM_THREADS / 32];
    pdl_trigger();
    pdl_wait();
    const int H = a.H;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const int64_t at = t * H;
        float mean0 = 0.0f, rstd0 = 0.0f, mean1 = 0.0f, rstd1 = 0.0f;
        for (int c = threadIdx.x; c < H; c += NORM_THREADS) row[c] = value(a.x[at + c]);
        if (a.post_w != nullptr) moments(row, H, a.kind, a.eps, part, mean0, rstd0);
        for (int c = threadIdx.x; c < H; c += NORM_THREADS) {
            float u = row[c];
            if (a.post_w != nullptr) {
                u = (u - mean0) * rstd0 * value(a.post_w[c]);
                if (a.post_b != nullptr) u += value(a.post_b[c]);
            }
            u *= a.scale * gate_at(a.gate, a.gate_form, t, c, H);
            if (a.residual != nullptr) u += value(a.residual[at + c]);
            row[c] = u;
            if (a.s != nullptr) put(a.s + at + c, u);
        }
        if (a.pre_w != nullptr) {
            moments(row, H, a.kind, a.eps, part, mean1, rstd1);
            for (int c = threadIdx.x; c < H; c += NORM_THREADS) {
                float y = (row[c] - mean1) * rstd1 * value(a.pre_w[c]);
                if (a.pre_b != nullptr) y += value(a.pre_b[c]);
                put(a.y + at + c, y);
            }
        }
        if (a.stats != nullptr && threadIdx.x == 0)
            reinterpret_cast<float4 *>(a.stats)[t] = make_float4(mean0, rstd0, mean1, rstd1);
    }
}

template <typename D> struct NormBwdArgs {
    const D *g_s, *g_y, *x, *s, *post_w, *post_b, *gate, *pre_w;
    const float *stats;
    int64_t T;
    int H, kind, gate_form;
    float scale;
    D *g_x, *g_residual, *g_gate;   // g_gate: a token's or an element's
    float *sums[NORM_SHARED];       // [NORM_PARTS,H] or NULL: post_w, post_b, pre_w, pre_b, gate
};

template <typename D> __global__ void __launch_bounds__(NORM_THREADS) k_block_norm_bwd(const NormBwdArgs<D> a)
{
    extern __shared__ float row[];
    __shared__ float part[NORM_THREADS / 32];
    pdl_trigger();
    pdl_wait();
    const int H = a.H;
    const float inv = 1.0f / static_cast<float>(H);
    const bool layer = a.kind == MP_NORM_LAYER;
    const auto sum = [&](int i, int c) -> float & { return a.sums[i][static_cast<int64_t>(blockIdx.x) * H + c]; };
    for (int i = 0; i < NORM_SHARED; ++i)
        if (a.sums[i] != nullptr)
            for (int c = threadIdx.x; c < H; c += NORM_THREADS) sum(i, c) = 0.0f;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const int64_t at = t * H;
        const float4 st = a.stats != nullptr ? reinterpret_cast<const float4 *>(a.stats)[t] : make_float4(0, 0, 0, 0);
        float flat = 0.0f, along = 0.0f;
        if (a.pre_w != nullptr) {
            for (int c = threadIdx.x; c < H; c += NORM_THREADS) {
                const float g = value(a.g_y[at + c]), hat = (value(a.s[at + c]) - st.z) * st.w;
                const float d = g * value(a.pre_w[c]);
                flat += d;
                along += d * hat;
                if (a.sums[2] != nullptr) sum(2, c) += g * hat;
                if (a.sums[3] != nullptr) sum(3, c) += g;
            }
            flat = layer ? cta_sum(flat, part) * inv : 0.0f;
            along = cta_sum(along, part) * inv;
        }
        float flat0 = 0.0f, along0 = 0.0f, gate_sum = 0.0f;
        for (int c = threadIdx.x; c < H; c += NORM_THREADS) {
            float total = a.g_s != nullptr ? value(a.g_s[at + c]) : 0.0f;
            if (a.pre_w != nullptr) {
                const float hat = (value(a.s[at + c]) - st.z) * st.w;
                total += st.w * (value(a.g_y[at + c]) * value(a.pre_w[c]) - flat - hat * along);
            }
            float g = a.scale * total;
            float hat = 0.0f;
            if (a.post_w != nullptr) hat = (value(a.x[at + c]) - st.x) * st.y;
            if (a.gate != nullptr) {
                float u = a.post_w != nullptr ? hat * value(a.post_w[c]) : value(a.x[at + c]);
                if (a.post_b != nullptr) u += value(a.post_b[c]);
                u *= g;
                g *= gate_at(a.gate, a.gate_form, t, c, H);
                if (a.gate_form == MP_GATE_ELEMENT && a.g_gate != nullptr) put(a.g_gate + at + c, u);
                if (a.sums[4] != nullptr) sum(4, c) += u;
                gate_sum += u;
            }
            if (a.g_residual != nullptr) put(a.g_residual + at + c, total);
            if (a.post_w != nullptr) {
                if (a.sums[0] != nullptr) sum(0, c) += g * hat;
                if (a.sums[1] != nullptr) sum(1, c) += g;
                g *= value(a.post_w[c]);
                flat0 += g;
                along0 += g * hat;
            }
            row[c] = g;
        }
        if (a.gate_form == MP_GATE_TOKEN && a.g_gate != nullptr) {
            gate_sum = cta_sum(gate_sum, part);
            if (threadIdx.x == 0) put(a.g_gate + t, gate_sum);
        }
        if (a.post_w != nullptr) {
            flat0 = layer ? cta_sum(flat0, part) * inv : 0.0f;
            along0 = cta_sum(along0, part) * inv;
        }
        if (a.g_x != nullptr)
            for (int c = threadIdx.x; c < H; c += NORM_THREADS) {
                float g = row[c];
                if (a.post_w != nullptr) g = st.y * (g - flat0 - (value(a.x[at + c]) - st.x) * st.y * along0);
                put(a.g_x + at + c, g);
            }
    }
}

struct NormSums {
    const float *sums[NORM_SHARED];
    void *out[NORM_SHARED];
};

// out[c] = the parts' sums in their order, in 64 bits: 152 values a column.
template <typename G> __global__ void __launch_bounds__(NORM_THREADS) k_norm_sums(const NormSums a, int parts, int H)
{
    pdl_trigger();
    pdl_wait();
    const float *from = a.sums[blockIdx.y];
    const int c = blockIdx.x * NORM_THREADS + threadIdx.x;
    if (c >= H) return;
    double v = 0.0;
#pragma unroll 8
    for (int i = 0; i < parts; ++i) v += from[static_cast<int64_t>(i) * H + c];
    put(static_cast<G *>(a.out[blockIdx.y]) + c, static_cast<float>(v));
}

mp_status_t norm_sizes(int64_t T, int32_t H, int32_t dtype, int32_t kind, int32_t gate_form, const void *gate,
                       float scale)
{
    if (T < 0 || H < 1 || dtype < MP_DTYPE_BF16 || dtype > MP_DTYPE_FP32 || kind < MP_NORM_RMS ||
        kind > MP_NORM_LAYER || gate_form < MP_GATE_NONE || gate_form > MP_GATE_ELEMENT)
        return MP_ERR_INVALID_ARG;
    if (T > 0 && (gate_form != MP_GATE_NONE) != (gate != nullptr)) return MP_ERR_INVALID_ARG;
    (void)scale;
    return H > MP_MAX_NORM_WIDTH || T > INT32_MAX ? MP_ERR_UNSUPPORTED : MP_OK;
}

template <typename K> mp_status_t allow_row(K kernel, int H)
{
    const cudaError_t err =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, MP_MAX_NORM_WIDTH * 4);
    (void)H;
    if (err == cudaSuccess) return MP_OK;
    set_last_cuda_error(err);
    return MP_ERR_CUDA;
}

template <typename D>
mp_status_t norm_fwd(const void *x, const void *residual, int64_t T, int32_t H, int32_t kind, float eps,
                     const void *post_w, const void *post_b, const void *gate, int32_t gate_form, float scale,
                     const void *pre_w, const void *pre_b, void *s, void *y, float *stats, cudaStream_t stream)
{
    NormArgs<D> a = {static_cast<const D *>(x), static_cast<const D *>(residual), static_cast<const D *>(post_w),
                     static_cast<const D *>(post_b), static_cast<const D *>(gate), static_cast<const D *>(pre_w),
                     static_cast<const D *>(pre_b), T, H, kind, gate_form, eps, scale, static_cast<D *>(s),
                     static_cast<D *>(y), stats};
    if (const mp_status_t st = allow_row(k_block_norm<D>, H); st != MP_OK) return st;
    const int64_t grid = T < 4 * NORM_PARTS ? T : 4 * NORM_PARTS;
    (void)launch_pdl(k_block_norm<D>, static_cast<unsigned>(grid), NORM_THREADS, H * sizeof(float), stream, a);
    return check_launch();
}

template <typename D>
mp_status_t norm_bwd(NormBwdArgs<D> a, const NormSums &shared, int vectors, int32_t grad_dtype, cudaStream_t stream)
{
    const int parts = static_cast<int>(a.T < NORM_PARTS ? a.T : NORM_PARTS);
    if (parts > 0) {
        if (const mp_status_t st = allow_row(k_block_norm_bwd<D>, a.H); st != MP_OK) return st;
        (void)launch_pdl(k_block_norm_bwd<D>, parts, NORM_THREADS, a.H * sizeof(float), stream, a);
    }
    if (vectors > 0) {
        const dim3 grid((a.H + NORM_THREADS - 1) / NORM_THREADS, vectors);
        if (grad_dtype == MP_DTYPE_FP32)
            (void)launch_pdl(k_norm_sums<float>, grid, NORM_THREADS, 0, stream, shared, parts, a.H);
        else
            (void)launch_pdl(k_norm_sums<D>, grid, NORM_THREADS, 0, stream, shared, parts, a.H);
    }
    return check_launch();
}

}  // namespace
}  // namespace mp

using namespace mp;

extern "C" mp_status_t mp_block_norm(const void *x, const void *residual, int64_t T, int32_t H, int32_t dtype,
                                     int32_t kind, float eps, const void *post_weight, const void *post_bias,
                                     const void *gate, int32_t gate_form, float scale, const void *pre_weight,
                                     const void *pre_bias, void *s, void *y, float *stats, mp_stream_t stream)
{
    if (const mp_status_t st = norm_sizes(T, H, dtype, kind, gate_form, gate, scale); st != MP_OK) return st;
    if (!(eps >= 0.0f)) return MP_ERR_INVALID_ARG;
    if (T == 0) return MP_OK;
    const bool as_is = residual == nullptr && post_weight == nullptr && gate == nullptr && scale == 1.0f;
    if (x == nullptr || (post_weight == nullptr && pre_weight == nullptr) ||
        (post_bias != nullptr && post_weight == nullptr) || (pre_bias != nullptr && pre_weight == nullptr) ||
        (y != nullptr) != (pre_weight != nullptr) || (s == nullptr && !as_is) || !aligned16(stats))
        return MP_ERR_INVALID_ARG;
    switch (dtype) {
    case MP_DTYPE_BF16:
        return norm_fwd<__nv_bfloat16>(x, residual, T, H, kind, eps, post_weight, post_bias, gate, gate_form, scale,
                                       pre_weight, pre_bias, s, y, stats, as_stream(stream));
    case MP_DTYPE_FP16:
        return norm_fwd<__half>(x, residual, T, H, kind, eps, post_weight, post_bias, gate, gate_form, scale,
                                pre_weight, pre_bias, s, y, stats, as_stream(stream));
    default:
        return norm_fwd<float>(x, residual, T, H, kind, eps, post_weight, post_bias, gate, gate_form, scale,
                               pre_weight, pre_bias, s, y, stats, as_stream(stream));
    }
}

extern "C" size_t mp_block_norm_bwd_workspace_size(int64_t T, int32_t H)
{
    if (T < 0 || H < 1 || H > MP_MAX_NORM_WIDTH || T > INT32_MAX) return 0;
    const size_t parts = static_cast<size_t>(T < NORM_PARTS ? T : NORM_PARTS);
    const size_t bytes = parts * NORM_SHARED * static_cast<size_t>(H) * sizeof(float);
    return bytes < 256 ? 256 : (bytes + 255) / 256 * 256;
}

extern "C" mp_status_t mp_block_norm_bwd(const void *g_s, const void *g_y, const void *x, const void *s,
                                         const float *stats, int64_t T, int32_t H, int32_t dtype, int32_t kind,
                                         const void *post_weight, const void *post_bias, const void *gate,
                                         int32_t gate_form, float scale, const void *pre_weight, void *g_x,
                                         void *g_residual, void *g_gate, void *g_post_weight, void *g_post_bias,
                                         void *g_pre_weight, void *g_pre_bias, int32_t grad_dtype, void *workspace,
                                         size_t workspace_bytes, mp_stream_t stream)
{
    if (const mp_status_t st = norm_sizes(T, H, dtype, kind, gate_form, gate, scale); st != MP_OK) return st;
    if (grad_dtype != dtype && grad_dtype != MP_DTYPE_FP32) return MP_ERR_INVALID_ARG;
    if ((g_gate != nullptr && gate_form == MP_GATE_NONE) ||
        (T > 0 && (post_weight == nullptr && pre_weight == nullptr)) ||
        (post_bias != nullptr && post_weight == nullptr && T > 0) ||
        (T > 0 && (g_post_weight != nullptr || g_post_bias != nullptr) && post_weight == nullptr) ||
        (T > 0 && (g_pre_weight != nullptr || g_pre_bias != nullptr) && pre_weight == nullptr))
        return MP_ERR_INVALID_ARG;
    if (T > 0 && (stats == nullptr || !aligned16(stats) || (pre_weight != nullptr && s == nullptr) ||
                  (pre_weight != nullptr) != (g_y != nullptr) || (pre_weight == nullptr && g_s == nullptr) ||
                  ((post_weight != nullptr || gate != nullptr) && x == nullptr)))
        return MP_ERR_INVALID_ARG;
    void *const shared[NORM_SHARED] = {g_post_weight, g_post_bias, g_pre_weight, g_pre_bias,
                                       gate_form == MP_GATE_CHANNEL ? g_gate : nullptr};
    NormSums n = {};
    float *sums[NORM_SHARED] = {};
    int vectors = 0;
    for (int i = 0; i < NORM_SHARED; ++i)
        if (shared[i] != nullptr) {
            sums[i] = static_cast<float *>(workspace) +
                      static_cast<size_t>(vectors) * static_cast<size_t>(T < NORM_PARTS ? T : NORM_PARTS) * H;
            n.sums[vectors] = sums[i];
            n.out[vectors++] = shared[i];
        }
    if (vectors > 0 && (workspace == nullptr || !aligned16(workspace) ||
                        workspace_bytes < mp_block_norm_bwd_workspace_size(T, H)))
        return MP_ERR_WORKSPACE;
    if (T == 0 && vectors == 0) return MP_OK;
    const auto run = [&](auto type) {
        typedef decltype(type) D;
        NormBwdArgs<D> a = {};
        a.g_s = static_cast<const D *>(g_s); a.g_y = static_cast<const D *>(g_y);
        a.x = static_cast<const D *>(x); a.s = static_cast<const D *>(s);
        a.post_w = static_cast<const D *>(post_weight); a.post_b = static_cast<const D *>(post_bias);
        a.gate = static_cast<const D *>(gate); a.pre_w = static_cast<const D *>(pre_weight);
        a.stats = stats; a.T = T; a.H = H; a.kind = kind; a.gate_form = gate_form; a.scale = scale;
        a.g_x = static_cast<D *>(g_x); a.g_residual = static_cast<D *>(g_residual);
        a.g_gate = gate_form == MP_GATE_CHANNEL ? nullptr : static_cast<D *>(g_gate);
        for (int i = 0; i < NORM_SHARED; ++i) a.sums[i] = sums[i];
        return norm_bwd<D>(a, n, vectors, grad_dtype, as_stream(stream));
    };
    switch (dtype) {
    case MP_DTYPE_BF16: return run(__nv_bfloat16());
    case MP_DTYPE_FP16: return run(__half());
    default: return run(0.0f);
    }
}
