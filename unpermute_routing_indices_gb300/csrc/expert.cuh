// What the experts' products share: activations and their derivatives, the
// 8-bit checkpoint of a row, the epilogues on 32 columns of a row, and the
// search for the expert of a tile.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace mp {

enum ExpertMode { FWD = 0, DGRAD = 1, WGRAD = 2 };

constexpr int EPI_COLS = 32;   // columns an epilogue step handles, and a checkpoint block

__host__ __device__ inline bool act_gated(int act) { return act >= MP_ACT_GEGLU; }
// The function on the gate (or on every column of an ungated product).
__host__ __device__ inline int act_inner(int act)
{
    return act == MP_ACT_GEGLU ? MP_ACT_GELU : act == MP_ACT_SWIGLU ? MP_ACT_SILU : act;
}
__host__ __device__ inline int ckpt_blocks(int n) { return (n + EPI_COLS - 1) / EPI_COLS; }

// ---------------------------------------------------------------------------
// Activations, in fp32.  The reciprocal is the approximate one (1 ulp), and so are
// the exponentials (2^-22), whose error grows with their argument by the rounding of
// that: silu 2^-20 of the value at z = -10, gelu, whose argument is a cubic in z, 2^-18 at
// z = -8, where it is 2^-70: below bf16's half step by far.
// ---------------------------------------------------------------------------

__device__ __forceinline__ float rcp_approx(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float exp2_approx(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// gelu in its tanh form is z * sigmoid(2u), u = sqrt(2/pi) (z + 0.044715 z^3):
// no difference of nearly equal numbers for negative z.  The exponential's argument
// is z (A + B z^2) with 1/ln 2 in both constants: three roundings and one
// instruction for 2^x (16,790 rows by 15 experts of 1,456 x 264 with expf 51 us, so 45).
constexpr float GELU_A = 1.5957691216057308f;    // 2 sqrt(2/pi)
constexpr float GELU_B = 0.044715f;
constexpr float GELU_A2 = -1.5957691216057308 * 1.4426950408889634;
constexpr float GELU_B2 = -1.5957691216057308 * 1.4426950408889634 * 0.044715;

// Past this bound gelu's derivative is 0 or 1 in fp32; NaN passes.
__device__ __forceinline__ float gelu_bounded(float z) { return z > 16.0f ? 16.0f : (z < -16.0f ? -16.0f : z); }

// act(z), and its derivative through `slope`.
template <int INNER> __device__ __forceinline__ float act_value_slope(float z, float &slope)
{
    if (INNER == MP_ACT_SILU) {
        const float s = rcp_approx(1.0f + __expf(-z)), a = z * s;
        slope = fmaf(a, 1.0f - s, s);
        return a;
    }
    if (INNER == MP_ACT_GELU) {
        const float c = gelu_bounded(z), cc = c * c;
        const float s = rcp_approx(1.0f + exp2_approx(c * fmaf(GELU_B2, cc, GELU_A2)));
        slope = fmaf(c * s * (1.0f - s), GELU_A * fmaf(3.0f * GELU_B, cc, 1.0f), s);
        return z * s;
    }
    if (INNER == MP_ACT_RELU) {
        slope = z > 0.0f ? 1.0f : 0.0f;
        return z < 0.0f ? 0.0f : z;
    }
    slope = 1.0f;
    return z;
}

template <int INNER> __device__ __forceinline__ float act_value(float z)
{
    float slope;
    return act_value_slope<INNER>(z, slope);
}

// ---------------------------------------------------------------------------
// 32 consecutive bf16 values of a row, on a 32-byte boundary.
// ---------------------------------------------------------------------------

__device__ __forceinline__ void unpack16(const u32x8 &v, float *f)
{
    float t[8];
    unpack(v.a, t);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = t[i];
    unpack(v.b, t);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[8 + i] = t[i];
}

__device__ __forceinline__ uint4 pack8(const float *f)
{
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

__device__ __forceinline__ unsigned low_bits(const void *p)
{
    return static_cast<unsigned>(reinterpret_cast<uintptr_t>(p)) & 31u;
}

__device__ __forceinline__ void load32(const mp_bf16_t *p, float (&f)[EPI_COLS])
{
    const u32x8 *q = reinterpret_cast<const u32x8 *>(p);
    const u32x8 v0 = ld_stream(q), v1 = ld_stream(q + 1);
    unpack16(v0, f);
    unpack16(v1, f + 16);
}

// fp32 weight gradients, added to what is there if `add`.
__device__ __forceinline__ void store32_f32(float *p, int n, const float (&f)[EPI_COLS], bool add)
{
    if (n >= EPI_COLS && (low_bits(p) & 15u) == 0) {
        float4 *q = reinterpret_cast<float4 *>(p);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float4 v = make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
            if (add) {
                const float4 o = q[j];
                v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
            }
            q[j] = v;
        }
    } else {
#pragma unroll
        for (int i = 0; i < EPI_COLS; ++i)
            if (i < n) p[i] = add ? p[i] + f[i] : f[i];
    }
}

// ---------------------------------------------------------------------------
// The 8-bit checkpoint: per row and 32 columns one power of two 2^(x-127), the
// smallest for which the block's largest finite magnitude is at most 448 of
// them, and e4m3 codes.  Powers of two make the scaling exact, so a value is
// rounded once, by at most half a step of e4m3 (2^-4 relative, 2^-10 of the
// unit below 2^-6 units).  What is not finite is stored as e4m3's NaN.
// ---------------------------------------------------------------------------

__device__ __forceinline__ int ckpt_exponent(float big)
{
    // big = m 2^k, 1 <= m < 2: 448 = 1.75 * 2^8, so the unit is 2^(k-8), or
    // one more where m > 1.75.
    const uint32_t u = __float_as_uint(big);
    const int x = static_cast<int>(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return x < 1 ? 1 : x;
}

__device__ __forceinline__ float pow2_biased(int x) { return __uint_as_float(static_cast<uint32_t>(x) << 23); }

__device__ __forceinline__ float finite_or_nan(float z) { return fmaf(z, 0.0f, z); }

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d)
{
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

__device__ __forceinline__ void e4m3x4_values(uint32_t u, float *f)
{
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(
            static_cast<__nv_fp8x2_storage_t>(u >> (16 * j)), __NV_E4M3);
        const float2 v = __half22float2(__half2(r));
        f[2 * j] = v.x;
        f[2 * j + 1] = v.y;
    }
}

__device__ __forceinline__ void ckpt_write32(uint8_t *codes, uint8_t *exponent, int n,
                                             const float (&z)[EPI_COLS])
{
    float big = 0.0f;
#pragma unroll
    for (int i = 0; i < EPI_COLS; ++i)
        if (i < n) big = fmaxf(big, fabsf(finite_or_nan(z[i])));   // fmaxf passes NaN over
    const int x = ckpt_exponent(big);
    const float inv = pow2_biased(254 - x);
    uint32_t c[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        c[j] = e4m3x4(finite_or_nan(z[4 * j]) * inv, finite_or_nan(z[4 * j + 1]) * inv,
                      finite_or_nan(z[4 * j + 2]) * inv, finite_or_nan(z[4 * j + 3]) * inv);
    const unsigned low = low_bits(codes);
    if (n >= EPI_COLS && low == 0) {
        st_row(reinterpret_cast<u32x8 *>(codes),
               u32x8{make_uint4(c[0], c[1], c[2], c[3]), make_uint4(c[4], c[5], c[6], c[7])});
    } else if (n >= EPI_COLS && (low & 7u) == 0) {
        uint2 *q = reinterpret_cast<uint2 *>(codes);
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = make_uint2(c[2 * j], c[2 * j + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < EPI_COLS; ++i)
            if (i < n) codes[i] = static_cast<uint8_t>(c[i / 4] >> (8 * (i % 4)));
    }
    *exponent = static_cast<uint8_t>(x);
}

__device__ __forceinline__ void ckpt_read32(const uint8_t *codes, const uint8_t *exponent, int n,
                                            float (&z)[EPI_COLS])
{
    const float unit = pow2_biased(ld_in(exponent));
    const unsigned low = low_bits(codes);
    uint32_t c[8];
    if (n >= EPI_COLS && low == 0) {
        const u32x8 v = ld_stream(reinterpret_cast<const u32x8 *>(codes));
        c[0] = v.a.x; c[1] = v.a.y; c[2] = v.a.z; c[3] = v.a.w;
        c[4] = v.b.x; c[5] = v.b.y; c[6] = v.b.z; c[7] = v.b.w;
    } else if (n >= EPI_COLS && (low & 7u) == 0) {
        const uint2 *q = reinterpret_cast<const uint2 *>(codes);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint2 v = ld_in(q + j);
            c[2 * j] = v.x;
            c[2 * j + 1] = v.y;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            c[j] = 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (4 * j + i < n) c[j] |= static_cast<uint32_t>(ld_in(codes + 4 * j + i)) << (8 * i);
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) e4m3x4_values(c[j], z + 4 * j);
#pragma unroll
    for (int i = 0; i < EPI_COLS; ++i) z[i] *= unit;
}

// ---------------------------------------------------------------------------
// Epilogues, on 32 columns of one row in fp32.  `W` reads and writes the bf16 rows of
// a warp, 32 consecutive ones, together: every lane calls, `valid` or not, with a
// row that exists to read from.
// ---------------------------------------------------------------------------

enum { TO_OUT = 0, TO_SECOND = 1 };   // the maps of a writer: out; z (FWD) or h (DGRAD)

struct ExpertEpi {
    int act, save;            // MP_ACT_*, MP_SAVE_*
    int cols;                 // columns of a part: of out (FWD), g_x's part (DGRAD), g_w (WGRAD)
    const mp_bf16_t *bias;    // FWD: [E, parts*cols] or NULL
    const mp_bf16_t *residual;
    mp_bf16_t *out;           // FWD: [R,cols]; DGRAD: [R, parts*cols]; WGRAD: [E,N,cols]
    void *z;                  // checkpoint [R, parts*cols]: written (FWD), read (DGRAD)
    uint8_t *z_exp;           // [R, parts*ckpt_blocks(cols)]
    mp_bf16_t *h;             // DGRAD: act(z) [R,cols] or NULL
    float *out_f32;           // WGRAD: fp32 gradient in place of `out`
    bool add;                 // WGRAD: add to out_f32 (and g_bias_f32)
    mp_bf16_t *g_bias;        // WGRAD: column sums of g [E,N] in bf16,
    float *g_bias_f32;        // or fp32; at most one of them given
    bool zero_rest;           // FWD, DGRAD (one part): rows of out that no expert has are zeroed
};

// Rows [first,last) of out, by thread `i` of `n`.
__device__ __forceinline__ void zero_rows(const ExpertEpi &p, int first, int last, int64_t i, int64_t n)
{
    mp_bf16_t *to = p.out + static_cast<int64_t>(first) * p.cols;
    const int64_t count = static_cast<int64_t>(last - first) * p.cols;
    if (p.cols % 8 == 0 && (reinterpret_cast<uintptr_t>(to) & 15u) == 0) {
        for (; i < count / 8; i += n) reinterpret_cast<uint4 *>(to)[i] = make_uint4(0, 0, 0, 0);
    } else {
        for (; i < count; i += n) to[i] = 0;
    }
}
// The rows of out that no expert has, of experts whose rows are [first,last).
__device__ __forceinline__ void zero_rest(const ExpertEpi &p, int first, int last, int R, int64_t i, int64_t n)
{
    zero_rows(p, 0, first, i, n);
    zero_rows(p, last, R, i, n);
}

template <typename W>
__device__ __forceinline__ void save32(const ExpertEpi &p, W &w, int64_t row, int part, int parts,
                                       int c, int n, bool valid, const float (&z)[EPI_COLS])
{
    if (p.save == MP_SAVE_BF16)
        w.put(static_cast<mp_bf16_t *>(p.z), static_cast<int64_t>(parts) * p.cols, TO_SECOND, row,
              static_cast<int64_t>(part) * p.cols + c, n, valid, z);
    else if (valid)
        ckpt_write32(static_cast<uint8_t *>(p.z) + (row * parts + part) * p.cols + c,
                     p.z_exp + (row * parts + part) * ckpt_blocks(p.cols) + c / EPI_COLS, n, z);
}

template <typename W>
__device__ __forceinline__ void read32(const ExpertEpi &p, W &w, int64_t row, int part, int parts, int c,
                                       int n, float (&z)[EPI_COLS])
{
    if (p.save == MP_SAVE_BF16)
        w.get(static_cast<const mp_bf16_t *>(p.z), static_cast<int64_t>(parts) * p.cols, row,
                              static_cast<int64_t>(part) * p.cols + c, n, z);
    else
        ckpt_read32(static_cast<const uint8_t *>(p.z) + (row * parts + part) * p.cols + c,
                    p.z_exp + (row * parts + part) * ckpt_blocks(p.cols) + c / EPI_COLS, n, z);
}

template <typename W>
__device__ __forceinline__ void add_bias32(W &w, const mp_bf16_t *b, int n, float (&z)[EPI_COLS])
{
    float f[EPI_COLS];
    w.get_shared(b, n, f);
#pragma unroll
    for (int i = 0; i < EPI_COLS; ++i) z[i] += f[i];
}

template <int INNER, bool GATED>
__device__ __forceinline__ void act32(float (&z)[EPI_COLS], const float (&u)[EPI_COLS])
{
#pragma unroll
    for (int i = 0; i < EPI_COLS; ++i) {
        z[i] = act_value<INNER>(z[i]);
        if (GATED) z[i] *= u[i];
    }
}

// z: the product's columns c..c+31 (of the gate when GATED, u then the others').
template <bool GATED, typename W>
__device__ __forceinline__ void epi_fwd(const ExpertEpi &p, W &w, int e, int64_t row, int c, int n,
                                        bool valid, float (&z)[EPI_COLS], float (&u)[EPI_COLS])
{
    constexpr int parts = GATED ? 2 : 1;
    if (p.bias != nullptr) {
        const mp_bf16_t *b = p.bias + static_cast<int64_t>(e) * parts * p.cols + c;
        add_bias32(w, b, n, z);
        if (GATED) add_bias32(w, b + p.cols, n, u);
    }
    if (p.save != MP_SAVE_NONE) {
        save32(p, w, row, 0, parts, c, n, valid, z);
        if (GATED) save32(p, w, row, 1, parts, c, n, valid, u);
    }
    switch (act_inner(p.act)) {
    case MP_ACT_SILU: act32<MP_ACT_SILU, GATED>(z, u); break;
    case MP_ACT_GELU: act32<MP_ACT_GELU, GATED>(z, u); break;
    case MP_ACT_RELU:
        if (!GATED) act32<MP_ACT_RELU, false>(z, u);
        break;
    default: break;
    }
    if (p.residual != nullptr) {
        float f[EPI_COLS];
        w.get(p.residual, p.cols, row, c, n, f);   // it may be out itself
#pragma unroll
        for (int i = 0; i < EPI_COLS; ++i) z[i] += f[i];
    }
    w.put(p.out, p.cols, TO_OUT, row, c, n, valid, z);
}

// g: the gradient of act's result.  The results replace their inputs: gated,
// z the gate's gradient, u the others', g act's result.
template <int INNER, bool GATED>
__device__ __forceinline__ void act_grad32(float (&g)[EPI_COLS], float (&z)[EPI_COLS], float (&u)[EPI_COLS])
{
#pragma unroll
    for (int i = 0; i < EPI_COLS; ++i) {
        float slope;
        const float a = act_value_slope<INNER>(z[i], slope);
        if (GATED) {
            z[i] = g[i] * u[i] * slope;
            const float o = u[i];
            u[i] = g[i] * a;
            g[i] = a * o;
        } else {
            z[i] = g[i] * slope;
            g[i] = a;
        }
    }
}

template <typename W>
__device__ __forceinline__ void epi_dgrad(const ExpertEpi &p, W &w, int64_t row, int c, int n,
                                          bool valid, float (&g)[EPI_COLS])
{
    if (p.act == MP_ACT_NONE) {
        w.put(p.out, p.cols, TO_OUT, row, c, n, valid, g);
        return;
    }
    float z[EPI_COLS], u[EPI_COLS];
    if (act_gated(p.act)) {
        read32(p, w, row, 0, 2, c, n, z);
        read32(p, w, row, 1, 2, c, n, u);
        if (p.act == MP_ACT_SWIGLU)
            act_grad32<MP_ACT_SILU, true>(g, z, u);
        else
            act_grad32<MP_ACT_GELU, true>(g, z, u);
        w.put(p.out, 2ll * p.cols, TO_OUT, row, c, n, valid, z);
        w.put(p.out, 2ll * p.cols, TO_OUT, row, static_cast<int64_t>(p.cols) + c, n, valid, u);
    } else {
        read32(p, w, row, 0, 1, c, n, z);
        switch (p.act) {
        case MP_ACT_SILU: act_grad32<MP_ACT_SILU, false>(g, z, u); break;
        case MP_ACT_GELU: act_grad32<MP_ACT_GELU, false>(g, z, u); break;
        default: act_grad32<MP_ACT_RELU, false>(g, z, u); break;
        }
        w.put(p.out, p.cols, TO_OUT, row, c, n, valid, z);
    }
    if (p.h != nullptr) w.put(p.h, p.cols, TO_SECOND, row, c, n, valid, g);
}

template <typename W>
__device__ __forceinline__ void epi_wgrad(const ExpertEpi &p, W &w, int64_t row, int c, int n,
                                          bool valid, const float (&g)[EPI_COLS])
{
    if (p.out_f32 == nullptr)
        w.put(p.out, p.cols, TO_OUT, row, c, n, valid, g);
    else if (valid)
        store32_f32(p.out_f32 + row * p.cols + c, n, g, p.add);
}

// ---------------------------------------------------------------------------
// Where each expert's rows start, clamped to [0,R] and made non-decreasing, so
// that no offset can lead outside a buffer; anything else sets a status bit.
// One warp fills start[0..E] and tiles[0..E] (tiles before each expert, of
// `tile_rows` rows).
// ---------------------------------------------------------------------------

// Each lane takes a run of entries, so that the two scans (largest so far, tiles so
// far) cross the warp once whatever E is.
__device__ __forceinline__ void expert_starts(const int32_t *offsets, int E, int R, int tile_rows,
                                              int lane, int *start, int *tiles, int32_t *status)
{
#pragma unroll 8
    for (int i = lane; i <= E; i += 32) start[i] = ld_in(offsets + i);
    __syncwarp();
    const int run = (E + 32) / 32, i0 = lane * run, i1 = min(i0 + run, E + 1);
    int high = 0;
    for (int i = i0; i < i1; ++i) high = max(high, min(start[i], R));
    int before = high;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(FULL_MASK, before, d);
        if (lane >= d) before = max(before, o);
    }
    before = __shfl_up_sync(FULL_MASK, before, 1);
    if (lane == 0) before = 0;
    // Entry i ends expert i - 1, whose rows start at the entry before it.
    bool bad = false;
    int prev = before, n = 0;
    for (int i = i0; i < i1; ++i) {
        const int given = start[i], v = max(prev, min(given, R));
        bad |= v != given;
        n += i > 0 ? (v - prev + tile_rows - 1) / tile_rows : 0;
        start[i] = v;
        tiles[i] = n;
        prev = v;
    }
    int sum = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(FULL_MASK, sum, d);
        if (lane >= d) sum += o;
    }
    sum -= n;
    for (int i = i0; i < i1; ++i) tiles[i] += sum;
    if (status != nullptr && __any_sync(FULL_MASK, bad) && lane == 0)
        or_status(status, MP_STATUS_BAD_OFFSETS);
}

// The expert of row tile t: tiles[e] <= t < tiles[e+1].
__device__ __forceinline__ int expert_of_tile(const int *tiles, int E, int t)
{
    int lo = 0, hi = E - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (tiles[mid + 1] > t)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}

// Launchers of the forms of the products (expert_*.cu).
struct ExpertCall {
    const mp_bf16_t *a, *b;   // FWD: x, w; DGRAD: g, w; WGRAD: g, x
    const int32_t *offsets;
    int R, E, N, K;           // w is [E,N,K]
    ExpertEpi epi;
    int32_t *status;
    cudaStream_t stream;
};

bool expert_by_tma(const ExpertCall &c, int mode);                   // TMA's rules hold
template <int MODE> mp_status_t expert_tc(const ExpertCall &c);
bool expert_few_takes(const ExpertCall &c);                          // FWD, few rows an expert
mp_status_t expert_few(const ExpertCall &c);

}  // namespace mp
