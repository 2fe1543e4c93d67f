// The experts' matrix products: argument checks, the choice of the kernel, and
// the gradient of the bias.
#include "expert.cuh"

namespace mp {
namespace {

constexpr int BIAS_THREADS = 256;

// g_bias[e,n] = sum over the expert's rows of g[row,n], in fp32; one warp takes
// every eighth row of 32 columns, and the eight sums are added in order.
__global__ void __launch_bounds__(BIAS_THREADS)
    k_expert_bias(const mp_bf16_t *__restrict__ g, const int32_t *__restrict__ offsets, int R,
                  int E, int N, mp_bf16_t *out, float *out_f32, bool add)
{
    pdl_trigger();
    pdl_wait();
    __shared__ int start[MP_MAX_EXPERTS + 1], tiles[MP_MAX_EXPERTS + 1];
    __shared__ float part[BIAS_THREADS / 32][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (warp == 0) expert_starts(offsets, E, R, 1, lane, start, tiles, nullptr);
    __syncthreads();
    const int e = blockIdx.y, n = blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (n < N)
        for (int r = start[e] + warp; r < start[e + 1]; r += BIAS_THREADS / 32) {
            float f[1];
            unpack(ld_stream(g + static_cast<int64_t>(r) * N + n), f);
            s += f[0];
        }
    part[warp][lane] = s;
    __syncthreads();
    if (warp != 0 || n >= N) return;
    for (int w = 1; w < BIAS_THREADS / 32; ++w) s += part[w][lane];
    const int64_t at = static_cast<int64_t>(e) * N + n;
    if (out_f32 != nullptr) {
        out_f32[at] = add ? out_f32[at] + s : s;
    } else {
        const float t[1] = {s};
        out[at] = pack(t);
    }
}

mp_status_t sizes_ok(int64_t R, int32_t E, int32_t N, int32_t K)
{
    if (R < 0 || E < 1 || N < 1 || K < 1) return MP_ERR_INVALID_ARG;
    if (E > MP_MAX_EXPERTS || R > INT32_MAX - 1024 || N > (1 << 22) || K > (1 << 22))
        return MP_ERR_UNSUPPORTED;
    return MP_OK;
}

template <int MODE> mp_status_t product(const ExpertCall &c)
{
    return expert_tc_takes<MODE>(c) ? expert_tc<MODE>(c) : expert_simt<MODE>(c);
}

bool act_ok(int32_t act) { return act >= MP_ACT_NONE && act <= MP_ACT_SWIGLU; }

}  // namespace
}  // namespace mp

using namespace mp;

extern "C" mp_status_t mp_expert_gemm(const mp_bf16_t *x, const mp_bf16_t *w,
                                      const int32_t *offsets, int64_t R, int32_t E, int32_t N,
                                      int32_t K, const mp_bf16_t *bias, int32_t act,
                                      const mp_bf16_t *residual, mp_bf16_t *out, int32_t save,
                                      void *z, uint8_t *z_exp, int32_t *dev_status,
                                      mp_stream_t stream)
{
    if (const mp_status_t s = sizes_ok(R, E, N, K); s != MP_OK) return s;
    if (!act_ok(act) || save < MP_SAVE_NONE || save > MP_SAVE_E4M3) return MP_ERR_INVALID_ARG;
    const bool gated = act_gated(act);
    if (gated && N % 2 != 0) return MP_ERR_INVALID_ARG;
    if (R == 0) return MP_OK;
    if (x == nullptr || w == nullptr || offsets == nullptr || out == nullptr ||
        (save != MP_SAVE_NONE && z == nullptr) || (save == MP_SAVE_E4M3 && z_exp == nullptr))
        return MP_ERR_INVALID_ARG;
    ExpertCall c = {};
    c.a = x; c.b = w; c.offsets = offsets;
    c.R = static_cast<int>(R); c.E = E; c.N = N; c.K = K;
    c.epi.act = act; c.epi.save = save; c.epi.cols = gated ? N / 2 : N;
    c.epi.bias = bias; c.epi.residual = residual; c.epi.out = out;
    c.epi.z = z; c.epi.z_exp = z_exp;
    c.status = dev_status;
    c.stream = as_stream(stream);
    return product<FWD>(c);
}

extern "C" mp_status_t mp_expert_dgrad(const mp_bf16_t *g, const mp_bf16_t *w,
                                       const int32_t *offsets, int64_t R, int32_t E, int32_t N,
                                       int32_t K, int32_t act, int32_t save, const void *z,
                                       const uint8_t *z_exp, mp_bf16_t *g_x, mp_bf16_t *h,
                                       int32_t *dev_status, mp_stream_t stream)
{
    if (const mp_status_t s = sizes_ok(R, E, N, K); s != MP_OK) return s;
    if (!act_ok(act)) return MP_ERR_INVALID_ARG;
    if (act == MP_ACT_NONE ? (save != MP_SAVE_NONE || h != nullptr)
                           : (save != MP_SAVE_BF16 && save != MP_SAVE_E4M3))
        return MP_ERR_INVALID_ARG;
    if (R == 0) return MP_OK;
    if (g == nullptr || w == nullptr || offsets == nullptr || g_x == nullptr ||
        (save != MP_SAVE_NONE && z == nullptr) || (save == MP_SAVE_E4M3 && z_exp == nullptr))
        return MP_ERR_INVALID_ARG;
    ExpertCall c = {};
    c.a = g; c.b = w; c.offsets = offsets;
    c.R = static_cast<int>(R); c.E = E; c.N = N; c.K = K;
    c.epi.act = act; c.epi.save = save; c.epi.cols = K;
    c.epi.out = g_x; c.epi.h = h;
    c.epi.z = const_cast<void *>(z); c.epi.z_exp = const_cast<uint8_t *>(z_exp);
    c.status = dev_status;
    c.stream = as_stream(stream);
    return product<DGRAD>(c);
}

extern "C" mp_status_t mp_expert_wgrad(const mp_bf16_t *g, const mp_bf16_t *x,
                                       const int32_t *offsets, int64_t R, int32_t E, int32_t N,
                                       int32_t K, int32_t dtype, int32_t accumulate, void *g_w,
                                       void *g_bias, int32_t *dev_status, mp_stream_t stream)
{
    if (const mp_status_t s = sizes_ok(R, E, N, K); s != MP_OK) return s;
    if ((dtype != MP_DTYPE_BF16 && dtype != MP_DTYPE_FP32) ||
        (accumulate != 0 && dtype != MP_DTYPE_FP32))
        return MP_ERR_INVALID_ARG;
    if (offsets == nullptr || g_w == nullptr || (R > 0 && (g == nullptr || x == nullptr)))
        return MP_ERR_INVALID_ARG;
    const bool f32 = dtype == MP_DTYPE_FP32;
    ExpertCall c = {};
    c.a = g; c.b = x; c.offsets = offsets;
    c.R = static_cast<int>(R); c.E = E; c.N = N; c.K = K;
    c.epi.cols = K;
    c.epi.out = f32 ? nullptr : static_cast<mp_bf16_t *>(g_w);
    c.epi.out_f32 = f32 ? static_cast<float *>(g_w) : nullptr;
    c.epi.add = accumulate != 0;
    c.status = dev_status;
    c.stream = as_stream(stream);
    const mp_status_t s = product<WGRAD>(c);
    if (s != MP_OK || g_bias == nullptr) return s;
    (void)launch_pdl(k_expert_bias, dim3((N + 31) / 32, E), BIAS_THREADS, 0, c.stream, g, offsets,
                     c.R, E, N, f32 ? nullptr : static_cast<mp_bf16_t *>(g_bias),
                     f32 ? static_cast<float *>(g_bias) : nullptr, c.epi.add);
    return check_launch();
}
