// mp_block_norm, mp_block_norm_bwd: checks of arguments, the choice of the form, and the
// last step of the gradients that rows share.
#include "norm.cuh"

namespace mp {
namespace {

struct NormSums {
    const float *sums[NORM_SHARED];
    void *out[NORM_SHARED];
};

constexpr int SUM_COLS = 32, SUM_ROWS = 16;

// A sum and what its roundings lost (Knuth's two-sum).
__device__ __forceinline__ void add_to(float2 &v, float p)
{
    const float t = __fadd_rn(v.x, p), z = __fsub_rn(t, v.x);
    v.y = __fadd_rn(v.y, __fadd_rn(__fsub_rn(v.x, __fsub_rn(t, z)), __fsub_rn(p, z)));
    v.x = t;
}

// out[c] = the CTAs' partial sums of column c, in pairs of fp32 and a fixed order: 16 threads a column,
// each every 16th of up to 152 of them, then the 16.  (In 64 bits, whose units are few, the
// gradient at one norm, 16,384 x 4,096, took 96 us in all.)
template <typename D> __global__ void __launch_bounds__(SUM_COLS *SUM_ROWS) k_norm_sums(const NormSums a, int parts, int H)
{
    __shared__ float2 part[SUM_ROWS][SUM_COLS];
    pdl_trigger();
    pdl_wait();
    const float *from = a.sums[blockIdx.y];
    const int col = threadIdx.x % SUM_COLS, row = threadIdx.x / SUM_COLS, c = blockIdx.x * SUM_COLS + col;
    float2 v = make_float2(0.0f, 0.0f);
    if (c < H) {
        constexpr int MOST = (NORM_PARTS + SUM_ROWS - 1) / SUM_ROWS;
        float p[MOST];
#pragma unroll
        for (int i = 0; i < MOST; ++i)
            p[i] = row + i * SUM_ROWS < parts ? from[static_cast<int64_t>(row + i * SUM_ROWS) * H + c] : 0.0f;
#pragma unroll
        for (int i = 0; i < MOST; ++i) add_to(v, p[i]);
    }
    part[row][col] = v;
    __syncthreads();
    if (row != 0 || c >= H) return;
#pragma unroll
    for (int i = 1; i < SUM_ROWS; ++i) {
        const float2 o = part[i][col];
        add_to(v, o.x);
        v.y = __fadd_rn(v.y, o.y);
    }
    norm_put(static_cast<D *>(a.out[blockIdx.y]) + c, isfinite(v.x) ? __fadd_rn(v.x, v.y) : v.x);
}

mp_status_t norm_sizes(int64_t T, int32_t H, int32_t dtype, int32_t kind, int32_t gate_form, const void *gate)
{
    if (T < 0 || H < 1 || dtype < MP_DTYPE_BF16 || dtype > MP_DTYPE_FP32 || kind < MP_NORM_RMS ||
        kind > MP_NORM_LAYER || gate_form < MP_GATE_NONE || gate_form > MP_GATE_ELEMENT)
        return MP_ERR_INVALID_ARG;
    if (T > 0 && (gate_form != MP_GATE_NONE) != (gate != nullptr)) return MP_ERR_INVALID_ARG;
    return H > MP_MAX_NORM_WIDTH || T > INT32_MAX ? MP_ERR_UNSUPPORTED : MP_OK;
}

size_t value_bytes(int32_t dtype) { return dtype == MP_DTYPE_FP32 ? 4 : 2; }

NormRows rows_of(const void *p, const NormCall &c, int32_t dtype)
{
    return {p, static_cast<int64_t>(reinterpret_cast<uintptr_t>(p)) +
                   c.T * c.H * static_cast<int64_t>(value_bytes(dtype))};
}

// Rows of whole 16-byte vectors, every tensor (NULL ones pass) on 16 bytes.
bool vectors(int32_t H, int32_t dtype, std::initializer_list<const void *> tensors)
{
    if (H * value_bytes(dtype) % 16 != 0) return false;
    for (const void *p : tensors)
        if (!aligned16(p)) return false;
    return true;
}

}  // namespace
}  // namespace mp

using namespace mp;

extern "C" mp_status_t mp_block_norm(const void *x, const void *residual, int64_t T, int32_t H, int32_t dtype,
                                     int32_t kind, float eps, const void *post_weight, const void *post_bias,
                                     const void *gate, int32_t gate_form, float scale, const void *pre_weight,
                                     const void *pre_bias, void *s, void *y, float *stats, int32_t *dev_status,
                                     mp_stream_t stream)
{
    if (const mp_status_t st = norm_sizes(T, H, dtype, kind, gate_form, gate); st != MP_OK) return st;
    if (!(eps >= 0.0f)) return MP_ERR_INVALID_ARG;
    if (T == 0) return MP_OK;
    const bool as_is = residual == nullptr && post_weight == nullptr && gate == nullptr && scale == 1.0f;
    if (x == nullptr || (post_weight == nullptr && pre_weight == nullptr) ||
        (post_bias != nullptr && post_weight == nullptr) || (pre_bias != nullptr && pre_weight == nullptr) ||
        (y != nullptr) != (pre_weight != nullptr) || (s == nullptr && !as_is) || (y != nullptr && s == y) ||
        !aligned16(stats))
        return MP_ERR_INVALID_ARG;
    NormCall c = {};
    c.T = T; c.H = H; c.kind = kind; c.gate_form = gate_form; c.eps = eps; c.scale = scale;
    c.x = rows_of(x, c, dtype);
    if (residual != nullptr) c.residual = rows_of(residual, c, dtype);
    if (gate_form == MP_GATE_ELEMENT) c.gate_rows = rows_of(gate, c, dtype);
    c.post_w = post_weight; c.post_b = post_bias; c.gate = gate; c.pre_w = pre_weight; c.pre_b = pre_bias;
    c.s_out = s; c.y = y; c.stats = stats; c.status = dev_status; c.stream = as_stream(stream);
    c.vec = vectors(H, dtype, {x, residual, gate_form == MP_GATE_TOKEN ? nullptr : gate, post_weight, post_bias,
                               pre_weight, pre_bias, s, y});
    return dtype == MP_DTYPE_BF16   ? norm_forward<__nv_bfloat16>(c)
           : dtype == MP_DTYPE_FP16 ? norm_forward<__half>(c)
                                    : norm_forward<float>(c);
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
                                         size_t workspace_bytes, int32_t *dev_status, mp_stream_t stream)
{
    if (const mp_status_t st = norm_sizes(T, H, dtype, kind, gate_form, gate); st != MP_OK) return st;
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
    // Rows are written one result after another, g_residual before x and the gate are read.
    const bool with_x = post_weight != nullptr || gate != nullptr;
    const void *const g_elements = gate_form == MP_GATE_ELEMENT ? g_gate : nullptr;
    if (g_residual != nullptr &&
        ((g_residual == g_x && (with_x || scale != 1.0f)) || g_residual == g_elements || (with_x && g_residual == x) ||
         (gate_form == MP_GATE_ELEMENT && g_residual == gate)))
        return MP_ERR_INVALID_ARG;
    if (g_elements != nullptr && g_elements == g_x) return MP_ERR_INVALID_ARG;
    void *const shared[NORM_SHARED] = {g_post_weight, g_post_bias, g_pre_weight, g_pre_bias,
                                       gate_form == MP_GATE_CHANNEL ? g_gate : nullptr};
    NormSums n = {};
    float *sums[NORM_SHARED] = {};
    int vectors_wanted = 0;
    for (int i = 0; i < NORM_SHARED; ++i)
        if (shared[i] != nullptr) {
            for (int k = 0; k < i; ++k)
                if (shared[k] == shared[i]) return MP_ERR_INVALID_ARG;
            sums[i] = static_cast<float *>(workspace) +
                      static_cast<size_t>(vectors_wanted) * static_cast<size_t>(T < NORM_PARTS ? T : NORM_PARTS) * H;
            n.sums[vectors_wanted] = sums[i];
            n.out[vectors_wanted++] = shared[i];
        }
    if (vectors_wanted > 0 && (workspace == nullptr || !aligned16(workspace) ||
                        workspace_bytes < mp_block_norm_bwd_workspace_size(T, H)))
        return MP_ERR_WORKSPACE;
    int parts = 0;
    if (T > 0) {
        NormCall c = {};
        c.T = T; c.H = H; c.kind = kind; c.gate_form = gate_form; c.scale = scale;
        if (g_s != nullptr) c.g_s = rows_of(g_s, c, dtype);
        if (pre_weight != nullptr) {
            c.g_y = rows_of(g_y, c, dtype);
            c.s = rows_of(s, c, dtype);
        }
        c.x = rows_of(x, c, dtype);
        if (gate_form == MP_GATE_ELEMENT) c.gate_rows = rows_of(gate, c, dtype);
        c.post_w = post_weight; c.post_b = post_bias; c.gate = gate; c.pre_w = pre_weight;
        c.stats = const_cast<float *>(stats);
        c.g_x = g_x; c.g_residual = g_residual;
        c.g_gate = gate_form == MP_GATE_CHANNEL ? nullptr : g_gate;
        for (int i = 0; i < NORM_SHARED; ++i) c.sums[i] = sums[i];
        c.status = dev_status; c.stream = as_stream(stream);
        c.vec = vectors(H, dtype, {g_s, g_y, with_x ? x : nullptr, pre_weight != nullptr ? s : nullptr,
                                   gate_form == MP_GATE_TOKEN ? nullptr : gate, post_weight, post_bias, pre_weight,
                                   g_x, g_residual, c.g_gate != nullptr && gate_form == MP_GATE_ELEMENT ? g_gate : nullptr});
        const mp_status_t st = dtype == MP_DTYPE_BF16   ? norm_backward<__nv_bfloat16>(c, parts)
                               : dtype == MP_DTYPE_FP16 ? norm_backward<__half>(c, parts)
                                                        : norm_backward<float>(c, parts);
        if (st != MP_OK) return st;
    }
    if (vectors_wanted == 0) return MP_OK;
    const dim3 grid((H + SUM_COLS - 1) / SUM_COLS, vectors_wanted);
    const cudaStream_t q = as_stream(stream);
    if (grad_dtype == MP_DTYPE_FP32)
        (void)launch_pdl(k_norm_sums<float>, grid, SUM_COLS * SUM_ROWS, 0, q, n, parts, H);
    else if (grad_dtype == MP_DTYPE_BF16)
        (void)launch_pdl(k_norm_sums<__nv_bfloat16>, grid, SUM_COLS * SUM_ROWS, 0, q, n, parts, H);
    else
        (void)launch_pdl(k_norm_sums<__half>, grid, SUM_COLS * SUM_ROWS, 0, q, n, parts, H);
    return check_launch();
}
