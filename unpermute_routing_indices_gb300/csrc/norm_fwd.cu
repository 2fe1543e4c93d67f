// The norms before and after a block (mp_block_norm): see norm.cuh for the layout.
//
//   u = norm(x) w_post + b_post, or x;  s = residual + scale gate u;  y = norm(s) w_pre + b_pre
//
// A group holds its row's values in registers from the first load to the last store, so that
// a row costs its bytes once; mean and deviation are sums over those registers, the deviation
// around the mean.
#include "norm.cuh"

namespace mp {
namespace {

struct NormArgs {
    NormRows x, residual, gate_rows;
    const void *post_w, *post_b, *gate, *pre_w, *pre_b;
    int64_t T;
    int H, kind, gate_form;
    float eps, scale;
    void *s, *y;
    float *stats;
};

// What the rows share, held as it is stored (C 4: read again for each row).
template <typename D, bool VEC, int C> struct Held {
    typedef NormGroup<D, VEC, C> G;
    const D *at;
    uint4 v[VEC && C < 4 ? G::VECS : 1];
    D e[!VEC && C < 4 ? G::N : 1];
    __device__ __forceinline__ void hold(const G &g, const void *p)
    {
        at = static_cast<const D *>(p);
        if (C == 4 || p == nullptr) return;
        if (VEC) {
#pragma unroll
            for (int i = 0; i < G::VECS; ++i) {
                const int c = (i * g.W + g.tid) * G::NV;
                v[VEC && C < 4 ? i : 0] = c < g.H ? *reinterpret_cast<const uint4 *>(at + c) : make_uint4(0, 0, 0, 0);
            }
        } else {
#pragma unroll
            for (int i = 0; i < G::N; ++i) {
                const int c = i * g.W + g.tid;
                e[!VEC && C < 4 ? i : 0] = c < g.H ? at[c] : D(0.0f);
            }
        }
    }
    __device__ __forceinline__ void get(const G &g, float (&f)[G::N]) const
    {
        if (C == 4) {
            g.load(at, f);
        } else if (VEC) {
#pragma unroll
            for (int i = 0; i < G::VECS; ++i) vec_values(v[VEC && C < 4 ? i : 0], f + i * G::NV, at);
        } else {
#pragma unroll
            for (int i = 0; i < G::N; ++i) f[i] = norm_value(e[!VEC && C < 4 ? i : 0]);
        }
    }
};

template <typename G>
__device__ __forceinline__ void moments(G &g, const float (&v)[G::N], int kind, float eps, float &mean, float &rstd)
{
    const float n = static_cast<float>(g.H);
    float t[1] = {0.0f};
    mean = 0.0f;
    if (kind == MP_NORM_LAYER) {
#pragma unroll
        for (int i = 0; i < G::N; ++i) t[0] += v[i];
        g.sums(t);
        mean = t[0] / n;
        t[0] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < G::N; ++i) {
        const float d = v[i] - mean;
        t[0] = g.in(i) ? fmaf(d, d, t[0]) : t[0];
    }
    g.sums(t);
    rstd = 1.0f / sqrtf(t[0] / n + eps);
}

template <typename D, bool VEC, int C>
__global__ void __launch_bounds__(C < 4 ? NORM_THREADS : 2 * NORM_THREADS, C == 1 ? 2 : 1)
    k_block_norm(const NormArgs a, const NormPlan p)
{
    typedef NormGroup<D, VEC, C> G;
    extern __shared__ __align__(16) uint8_t smem[];
    pdl_trigger();
    pdl_wait();
    G g;
    g.W = p.W; g.H = a.H;
    g.group = threadIdx.x / p.W;
    g.tid = threadIdx.x - g.group * p.W;
    g.red = reinterpret_cast<float *>(smem) + (p.W > 32 ? g.group * G::RED : 0);
    const bool with_gate = a.gate_rows.at != nullptr, with_residual = a.residual.at != nullptr;
    const int tensors = 1 + with_residual + with_gate;
    uint8_t *const ring = smem + (p.W > 32 ? p.R : 1) * G::RED * 4 +
                          static_cast<size_t>(g.group) * p.stages * tensors * p.pitch;
    const int64_t step = static_cast<int64_t>(gridDim.x) * p.R, first = static_cast<int64_t>(blockIdx.x) * p.R;
    const auto fetch = [&](int64_t t, uint8_t *slot) {
        if (t < a.T) {
            g.fetch(a.x, t, slot);
            if (with_residual) g.fetch(a.residual, t, slot + p.pitch);
            if (with_gate) g.fetch(a.gate_rows, t, slot + (tensors - 1) * p.pitch);
        }
        cp_commit();
    };
    if (G::STAGED)
        for (int i = 0; i < p.stages; ++i) fetch(first + i * step + g.group, ring + i * tensors * p.pitch);
    Held<D, VEC, C> post_w, post_b, gate, pre_w, pre_b;
    post_w.hold(g, a.post_w);
    post_b.hold(g, a.post_b);
    gate.hold(g, a.gate_form == MP_GATE_CHANNEL ? a.gate : nullptr);
    pre_w.hold(g, a.pre_w);
    pre_b.hold(g, a.pre_b);
    // A token's gate, read one row ahead.
    const auto gate_of = [&](int64_t t) {
        return a.gate_form == MP_GATE_TOKEN && t < a.T ? norm_value(static_cast<const D *>(a.gate)[t]) : 1.0f;
    };
    float next_gate = gate_of(first + g.group);
    int at = 0;
    for (int64_t t0 = first; t0 < a.T; t0 += step) {   // the same count for every group
        const int64_t t = t0 + g.group;
        const bool there = t < a.T;
        uint8_t *const slot = ring + at * tensors * p.pitch;
        if (G::STAGED) {
            cp_wait(p.stages - 1);
            if (!VEC) g.barrier();
        }
        float v[G::N], w[G::N];
        float mean0 = 0.0f, rstd0 = 0.0f, mean1 = 0.0f, rstd1 = 0.0f;
        const float scale = a.scale * next_gate;
        next_gate = gate_of(t + step);
        if (there) {
            g.load(g.row(a.x, t, slot), v);
        } else {
#pragma unroll
            for (int i = 0; i < G::N; ++i) v[i] = 0.0f;
        }
        if (a.post_w != nullptr) {
            moments(g, v, a.kind, a.eps, mean0, rstd0);
            post_w.get(g, w);
#pragma unroll
            for (int i = 0; i < G::N; ++i) v[i] = (v[i] - mean0) * rstd0 * w[i];
            if (a.post_b != nullptr) {
                post_b.get(g, w);
#pragma unroll
                for (int i = 0; i < G::N; ++i) v[i] += w[i];
            }
        }
        if (a.gate_form == MP_GATE_CHANNEL) {
            gate.get(g, w);
#pragma unroll
            for (int i = 0; i < G::N; ++i) v[i] *= w[i];
        } else if (with_gate && there) {
            g.load(g.row(a.gate_rows, t, slot + (tensors - 1) * p.pitch), w);
#pragma unroll
            for (int i = 0; i < G::N; ++i) v[i] *= w[i];
        }
        if (with_residual && there) {
            g.load(g.row(a.residual, t, slot + p.pitch), w);
#pragma unroll
            for (int i = 0; i < G::N; ++i) v[i] = fmaf(scale, v[i], w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < G::N; ++i) v[i] *= scale;
        }
        // The row has been read: its slot takes the one `stages` steps on.
        if (G::STAGED) {
            if (!VEC) g.barrier();
            fetch(t + p.stages * step, slot);
            at = at + 1 == p.stages ? 0 : at + 1;
        }
        if (a.s != nullptr && there) g.store(static_cast<D *>(a.s) + t * a.H, v);
        if (a.pre_w != nullptr) {
            moments(g, v, a.kind, a.eps, mean1, rstd1);
            pre_w.get(g, w);
#pragma unroll
            for (int i = 0; i < G::N; ++i) v[i] = (v[i] - mean1) * rstd1 * w[i];
            if (a.pre_b != nullptr) {
                pre_b.get(g, w);
#pragma unroll
                for (int i = 0; i < G::N; ++i) v[i] += w[i];
            }
            if (there) g.store(static_cast<D *>(a.y) + t * a.H, v);
        }
        if (a.stats != nullptr && g.tid == 0 && there)
            reinterpret_cast<float4 *>(a.stats)[t] = make_float4(mean0, rstd0, mean1, rstd1);
    }
    if (G::STAGED) cp_wait(0);
}

template <typename D, bool VEC, int C> mp_status_t forward(const NormCall &c)
{
    static std::atomic<uint64_t> allowed{0};
    const int tensors = 1 + (c.residual.at != nullptr) + (c.gate_rows.at != nullptr);
    const NormArgs a = {c.x, c.residual, c.gate_rows, c.post_w, c.post_b, c.gate, c.pre_w, c.pre_b, c.T, c.H,
                        c.kind, c.gate_form, c.eps, c.scale, c.s_out, c.y, c.stats};
    int grid;
    return norm_launch(k_block_norm<D, VEC, C>, allowed, norm_plan<D>(c.T, c.H, C, tensors, 0, C == 1), C == 1, c.T,
                       c.stream, grid, a);
}

}  // namespace

template <typename D> mp_status_t norm_forward(const NormCall &c)
{
    if (c.H <= 8 * NORM_THREADS) return c.vec ? forward<D, true, 1>(c) : forward<D, false, 1>(c);
    if (c.H <= 16 * NORM_THREADS) return c.vec ? forward<D, true, 2>(c) : forward<D, false, 2>(c);
    return c.vec ? forward<D, true, 4>(c) : forward<D, false, 4>(c);
}
template mp_status_t norm_forward<__nv_bfloat16>(const NormCall &);
template mp_status_t norm_forward<__half>(const NormCall &);
template mp_status_t norm_forward<float>(const NormCall &);

}  // namespace mp
