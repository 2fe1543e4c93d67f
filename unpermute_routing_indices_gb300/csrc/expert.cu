// The experts' matrix products: argument checks, the choice of the kernel, and
// the gradient of the bias.
#include <type_traits>

#include "expert.cuh"

namespace mp {
namespace {

constexpr int BIAS_THREADS = 256, BIAS_WARPS = BIAS_THREADS / 32;

// g_bias[e,n] = sum over the expert's rows of g[row,n], in fp32.  A CTA owns 32 V
// columns of one expert, V = 8 (16-byte loads) where rows are aligned to it; each
// warp takes every eighth row, four of them in flight, and the eight sums are
// added in order.  The weight gradient makes these sums itself where TMA reads its
// operands; this serves the others, and biases whose weights want no gradient.
template <int V>
__global__ void __launch_bounds__(BIAS_THREADS)
    k_expert_bias(const mp_bf16_t *__restrict__ g, const int32_t *__restrict__ offsets, int R,
                  int E, int N, mp_bf16_t *out, float *out_f32, bool add)
{
    pdl_trigger();
    pdl_wait();
    __shared__ float part[BIAS_WARPS][32 * V];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = blockIdx.y;
    // The clamped offsets of this expert: the largest up to each.
    int a = 0, b = 0;
#pragma unroll 8
    for (int i = lane; i <= e + 1; i += 32) {
        const int v = min(max(__ldg(offsets + i), 0), R);
        b = max(b, v);
        if (i <= e) a = max(a, v);
    }
    a = __reduce_max_sync(FULL_MASK, a);
    b = __reduce_max_sync(FULL_MASK, b);
    const int n0 = blockIdx.x * 32 * V, n = n0 + lane * V;
    float s[V] = {};
    if (n < N) {
        typedef typename std::conditional<V == 8, uint4, uint16_t>::type Vec;
        const Vec *p = reinterpret_cast<const Vec *>(g + n);
        const int64_t pitch = N / V;
        int r = a + warp;
        for (; r + 3 * BIAS_WARPS < b; r += 4 * BIAS_WARPS) {
            Vec v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = ld_stream(p + (r + q * BIAS_WARPS) * pitch);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float f[V];
                unpack(v[q], f);
#pragma unroll
                for (int i = 0; i < V; ++i) s[i] += f[i];
            }
        }
        for (; r < b; r += BIAS_WARPS) {
            float f[V];
            unpack(ld_stream(p + r * pitch), f);
#pragma unroll
            for (int i = 0; i < V; ++i) s[i] += f[i];
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) part[warp][lane * V + i] = s[i];
    __syncthreads();
    if (threadIdx.x >= 32 * V || n0 + static_cast<int>(threadIdx.x) >= N) return;
    float t = part[0][threadIdx.x];
    for (int w = 1; w < BIAS_WARPS; ++w) t += part[w][threadIdx.x];
    const int64_t at = static_cast<int64_t>(e) * N + n0 + threadIdx.x;
    if (out_f32 != nullptr) {
        out_f32[at] = add ? out_f32[at] + t : t;
    } else {
        const float f[1] = {t};
        out[at] = pack(f);
    }
}

mp_status_t sizes_ok(int64_t R, int32_t E, int32_t N, int32_t K)
{
    if (R < 0 || E < 1 || N < 1 || K < 1) return MP_ERR_INVALID_ARG;
    if (E > MP_MAX_EXPERTS || R > INT32_MAX - 1024 || N > (1 << 22) || K > (1 << 22))
        return MP_ERR_UNSUPPORTED;
    return MP_OK;
}

// g_bias of c.N columns, in bf16 or fp32 (added to if c.epi.add).
mp_status_t bias_grad(const mp_bf16_t *g, const ExpertCall &c, mp_bf16_t *out, float *out_f32)
{
    if (c.N % 8 == 0 && aligned16(g))
        (void)launch_pdl(k_expert_bias<8>, dim3((c.N + 255) / 256, c.E), BIAS_THREADS, 0, c.stream, g,
                         c.offsets, c.R, c.E, c.N, out, out_f32, c.epi.add);
    else
        (void)launch_pdl(k_expert_bias<1>, dim3((c.N + 31) / 32, c.E), BIAS_THREADS, 0, c.stream, g,
                         c.offsets, c.R, c.E, c.N, out, out_f32, c.epi.add);
    return check_launch();
}

// g_w as c.epi has it, and g_bias (NULL: not wanted): within the product, or by a
// kernel of its own where the load warps read the operands.
mp_status_t weight_grad(ExpertCall &c, void *g_bias, bool f32)
{
    mp_bf16_t *b = f32 ? nullptr : static_cast<mp_bf16_t *>(g_bias);
    float *b32 = f32 ? static_cast<float *>(g_bias) : nullptr;
    const bool within = expert_by_tma(c, WGRAD);
    if (within) {
        c.epi.g_bias = b;
        c.epi.g_bias_f32 = b32;
    }
    const mp_status_t s = expert_tc<WGRAD>(c);
    return s != MP_OK || within || g_bias == nullptr ? s : bias_grad(c.a, c, b, b32);
}

bool act_ok(int32_t act) { return act >= MP_ACT_NONE && act <= MP_ACT_SWIGLU; }

}  // namespace
}  // namespace mp

using namespace mp;

namespace {

// mp_expert_gemm and mp_expert_dgrad; zero_rest: rows of the result that no expert
// has are zeroed.
mp_status_t gemm(const mp_bf16_t *x, const mp_bf16_t *w, const int32_t *offsets, int64_t R, int32_t E,
                 int32_t N, int32_t K, const mp_bf16_t *bias, int32_t act, const mp_bf16_t *residual,
                 mp_bf16_t *out, int32_t save, void *z, uint8_t *z_exp, bool zero_rest,
                 int32_t *dev_status, mp_stream_t stream)
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
    c.epi.zero_rest = zero_rest;
    c.status = dev_status;
    c.stream = as_stream(stream);
    if (expert_few_takes(c)) return expert_few(c);
    return expert_tc<FWD>(c);
}

mp_status_t dgrad(const mp_bf16_t *g, const mp_bf16_t *w, const int32_t *offsets, int64_t R, int32_t E,
                  int32_t N, int32_t K, int32_t act, int32_t save, const void *z,
                  const uint8_t *z_exp, mp_bf16_t *g_x, mp_bf16_t *h, bool zero_rest,
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
    c.epi.zero_rest = zero_rest;
    c.status = dev_status;
    c.stream = as_stream(stream);
    return expert_tc<DGRAD>(c);
}

}  // namespace

extern "C" mp_status_t mp_expert_gemm(const mp_bf16_t *x, const mp_bf16_t *w,
                                      const int32_t *offsets, int64_t R, int32_t E, int32_t N,
                                      int32_t K, const mp_bf16_t *bias, int32_t act,
                                      const mp_bf16_t *residual, mp_bf16_t *out, int32_t save,
                                      void *z, uint8_t *z_exp, int32_t *dev_status,
                                      mp_stream_t stream)
{
    return gemm(x, w, offsets, R, E, N, K, bias, act, residual, out, save, z, z_exp, false, dev_status, stream);
}

extern "C" mp_status_t mp_expert_dgrad(const mp_bf16_t *g, const mp_bf16_t *w,
                                       const int32_t *offsets, int64_t R, int32_t E, int32_t N,
                                       int32_t K, int32_t act, int32_t save, const void *z,
                                       const uint8_t *z_exp, mp_bf16_t *g_x, mp_bf16_t *h,
                                       int32_t *dev_status, mp_stream_t stream)
{
    return dgrad(g, w, offsets, R, E, N, K, act, save, z, z_exp, g_x, h, false, dev_status, stream);
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
    return weight_grad(c, g_bias, f32);
}

extern "C" mp_status_t mp_expert_mlp(const mp_bf16_t *x, const mp_bf16_t *w1, const mp_bf16_t *b1,
                                     const mp_bf16_t *w2, const mp_bf16_t *b2,
                                     const int32_t *offsets, int64_t R, int32_t E, int32_t H,
                                     int32_t F, int32_t O, int32_t act, mp_bf16_t *h, mp_bf16_t *y,
                                     int32_t save, void *z, uint8_t *z_exp, int32_t *dev_status,
                                     mp_stream_t stream)
{
    if (!act_ok(act) || act == MP_ACT_NONE || F < 1 || F > (1 << 21)) return MP_ERR_INVALID_ARG;
    if (const mp_status_t s = sizes_ok(R, E, O, F); s != MP_OK) return s;
    if (R > 0 && (h == nullptr || w2 == nullptr || y == nullptr)) return MP_ERR_INVALID_ARG;
    const mp_status_t s = gemm(x, w1, offsets, R, E, act_gated(act) ? 2 * F : F, H, b1, act, nullptr, h, save,
                               z, z_exp, false, dev_status, stream);
    if (s != MP_OK) return s;
    return gemm(h, w2, offsets, R, E, O, F, b2, MP_ACT_NONE, nullptr, y, MP_SAVE_NONE, nullptr, nullptr, true,
                dev_status, stream);
}

extern "C" mp_status_t mp_expert_mlp_bwd(const mp_bf16_t *g_y, const mp_bf16_t *x,
                                         const mp_bf16_t *w1, const mp_bf16_t *w2,
                                         const int32_t *offsets, int64_t R, int32_t E, int32_t H,
                                         int32_t F, int32_t O, int32_t act, int32_t save,
                                         const void *z, const uint8_t *z_exp, mp_bf16_t *g_z,
                                         mp_bf16_t *h, mp_bf16_t *g_x, mp_bf16_t *g_w1,
                                         mp_bf16_t *g_b1, mp_bf16_t *g_w2, mp_bf16_t *g_b2,
                                         int32_t *dev_status, mp_stream_t stream)
{
    if (!act_ok(act) || act == MP_ACT_NONE || F < 1 || F > (1 << 21)) return MP_ERR_INVALID_ARG;
    const int32_t P = act_gated(act) ? 2 * F : F;
    for (const int32_t n : {H, O})
        if (const mp_status_t s = sizes_ok(R, E, P, n); s != MP_OK) return s;
    if (offsets == nullptr || (R > 0 && (g_y == nullptr || x == nullptr || g_z == nullptr)) ||
        (R > 0 && ((g_w2 != nullptr && h == nullptr) || (g_x != nullptr && w1 == nullptr))))
        return MP_ERR_INVALID_ARG;
    mp_status_t s = mp_expert_dgrad(g_y, w2, offsets, R, E, O, F, act, save, z, z_exp, g_z, h,
                                    dev_status, stream);
    if (s == MP_OK && g_w2 != nullptr)
        s = mp_expert_wgrad(g_y, h, offsets, R, E, O, F, MP_DTYPE_BF16, 0, g_w2, g_b2, dev_status, stream);
    if (s == MP_OK && g_w1 != nullptr)
        s = mp_expert_wgrad(g_z, x, offsets, R, E, P, H, MP_DTYPE_BF16, 0, g_w1, g_b1, dev_status, stream);
    // A bias's gradient without its weights'.
    ExpertCall c = {};
    c.offsets = offsets;
    c.R = static_cast<int>(R); c.E = E;
    c.stream = as_stream(stream);
    c.N = O;
    if (s == MP_OK && g_b2 != nullptr && g_w2 == nullptr) s = bias_grad(g_y, c, g_b2, nullptr);
    c.N = P;
    if (s == MP_OK && g_b1 != nullptr && g_w1 == nullptr) s = bias_grad(g_z, c, g_b1, nullptr);
    if (s != MP_OK || g_x == nullptr || R == 0) return s;
    return dgrad(g_z, w1, offsets, R, E, P, H, MP_ACT_NONE, MP_SAVE_NONE, nullptr, nullptr, g_x, nullptr, true,
                 dev_status, stream);
}
