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
    NormInputs in;
    const void *post_w, *post_b, *gate, *pre_w, *pre_b;
    int64_t T;
    int H, kind, gate_form;
    float eps, scale;
    void *s, *y;
    float *stats;
    int32_t *status;
};
enum { ROW_X, ROW_RESIDUAL, ROW_GATE };

template <typename G>
__device__ __forceinline__ void moments(G &g, const f2 (&v)[G::N2], int kind, float eps, float inv, float &mean,
                                        float &rstd)
{
    float t[1];
    f2 sum = 0ull;
    mean = 0.0f;
    if (kind == MP_NORM_LAYER) {
#pragma unroll
        for (int i = 0; i < G::N2; ++i) sum = add2(sum, v[i]);
        t[0] = sum2(sum);
        g.sums(t);
        mean = t[0] * inv;
        sum = 0ull;
        const f2 off = pair(-mean, -mean);
#pragma unroll
        for (int i = 0; i < G::N2; ++i) {
            const f2 d = g.inside(i, add2(v[i], off));
            sum = fma2(d, d, sum);
        }
    } else {   // what is past the row's end is 0
#pragma unroll
        for (int i = 0; i < G::N2; ++i) sum = fma2(v[i], v[i], sum);
    }
    t[0] = sum2(sum);
    g.sums(t);
    rstd = __frsqrt_rn(fmaf(t[0], inv, eps));
}

// (v - mean) rstd w + b
template <typename G, typename D>
__device__ __forceinline__ void normalise(const G &g, f2 (&v)[G::N2], bool layer, float mean, float rstd, const D *w,
                                          const D *b, bool with_b)
{
    f2 t[G::N2];
    g.load_shared(w, t);
    const f2 off = pair(-mean, -mean), r = pair(rstd, rstd);
    if (layer) {
#pragma unroll
        for (int i = 0; i < G::N2; ++i) v[i] = add2(v[i], off);
    }
#pragma unroll
    for (int i = 0; i < G::N2; ++i) v[i] = mul2(mul2(v[i], r), t[i]);
    if (with_b) {
        g.load_shared(b, t);
#pragma unroll
        for (int i = 0; i < G::N2; ++i) v[i] = add2(v[i], t[i]);
    }
}

template <typename D, int M, int C>
__global__ void __launch_bounds__(C < 4 ? NORM_THREADS : 2 * NORM_THREADS, C < 4 ? 2 : 1)
    k_block_norm(const NormArgs a, const NormPlan p)
{
    typedef NormGroup<D, M, C> G;
    extern __shared__ __align__(16) uint8_t smem[];
    pdl_trigger();
    pdl_wait();
    G g;
    const int H = a.H;
    g.begin(smem, p.W, p.R, H);
    const bool with_gate = a.in.slot[ROW_GATE] >= 0, with_residual = a.in.slot[ROW_RESIDUAL] >= 0;
    const int slot_bytes = a.in.tensors * p.pitch;
    uint8_t *const rings = smem + G::head(p.W, p.R);
    uint8_t *const ring = rings + static_cast<size_t>(g.group) * p.stages * slot_bytes;
    const uint32_t T = static_cast<uint32_t>(a.T), step = gridDim.x * p.R, first = blockIdx.x * p.R;
    // What the rows share, in shared memory behind the slots: registers are short.
    uint8_t *held = rings + static_cast<size_t>(p.R) * p.stages * slot_bytes;
    const auto hold = [&](const void *v) {
        if constexpr (G::STAGED) {
            const D *const to = reinterpret_cast<const D *>(held);
            if (v != nullptr) {
                g.hold(static_cast<const D *>(v), held);
                held += p.held;
            }
            return to;
        } else {
            return static_cast<const D *>(v);
        }
    };
    const D *const post_w = hold(a.post_w), *const post_b = hold(a.post_b);
    const bool by_channel = a.gate_form == MP_GATE_CHANNEL;
    const D *const channel = hold(by_channel ? a.gate : nullptr);
    const D *const pre_w = hold(a.pre_w), *const pre_b = hold(a.pre_b);
    cp_commit();
    if (G::STAGED)
        for (int i = 0; i < p.stages; ++i) g.template fetch<5>(a.in, first + i * step + g.group, T, ring + i * slot_bytes, p.pitch, i);
    // A token's gate, read one row ahead.
    const auto gate_of = [&](uint32_t t) {
        return a.gate_form == MP_GATE_TOKEN && t < T ? norm_value(static_cast<const D *>(a.gate)[t]) : 1.0f;
    };
    float next_gate = gate_of(first + g.group);
    const bool layer = a.kind == MP_NORM_LAYER;
    const float inv = 1.0f / static_cast<float>(H);
    // The oldest copies are those of what the rows share.
    if (M == ROWS_BULK)
        cp_wait(0);
    else
        cp_wait(p.stages);
    __syncthreads();
    int at = 0;
    for (uint32_t t0 = first; t0 < T; t0 += step) {   // the same count for every group
        const uint32_t t = t0 + g.group;
        const bool there = t < T;
        const uint64_t row = static_cast<uint64_t>(t) * static_cast<uint32_t>(H);
        uint8_t *const slot = ring + at * slot_bytes;
        g.arrived(at, p.stages, there);
        f2 v[G::N2], w[G::N2];
        float mean0 = 0.0f, rstd0 = 0.0f, mean1 = 0.0f, rstd1 = 0.0f;
        const float scale = a.scale * next_gate;
        next_gate = gate_of(t + step);
#pragma unroll
        for (int i = 0; i < G::N2; ++i) v[i] = 0ull;
        if (there) g.load(g.row(a.in.rows[ROW_X], t, slot), v);
        if (a.post_w != nullptr) {
            moments(g, v, a.kind, a.eps, inv, mean0, rstd0);
            normalise(g, v, layer, mean0, rstd0, post_w, post_b, a.post_b != nullptr);
        }
        if (by_channel) {
            g.load_shared(channel, w);
#pragma unroll
            for (int i = 0; i < G::N2; ++i) v[i] = mul2(v[i], w[i]);
        } else if (with_gate && there) {
            g.load(g.row(a.in.rows[ROW_GATE], t, slot + a.in.slot[ROW_GATE] * p.pitch), w);
#pragma unroll
            for (int i = 0; i < G::N2; ++i) v[i] = mul2(v[i], w[i]);
        }
        const f2 by = pair(scale, scale);
        if (with_residual && there) {
            g.load(g.row(a.in.rows[ROW_RESIDUAL], t, slot + a.in.slot[ROW_RESIDUAL] * p.pitch), w);
#pragma unroll
            for (int i = 0; i < G::N2; ++i) v[i] = fma2(by, v[i], w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < G::N2; ++i) v[i] = mul2(v[i], by);
        }
        // The row has been read (by everyone, after the next sum or a barrier): its slot takes the
        // one `stages` steps on.
        const auto refill = [&]() {
            if (G::STAGED) {
                g.template fetch<5>(a.in, t + p.stages * step, T, slot, p.pitch, at);
                at = g.after(at, p.stages);
            }
        };
        if (M == ROWS_VEC) refill();
        if (a.s != nullptr && there) g.store(static_cast<D *>(a.s) + row, v);
        if (a.pre_w != nullptr) {
            moments(g, v, a.kind, a.eps, inv, mean1, rstd1);
            if (M == ROWS_BULK) refill();
            normalise(g, v, layer, mean1, rstd1, pre_w, pre_b, a.pre_b != nullptr);
            if (there) g.store(static_cast<D *>(a.y) + row, v);
        }
        if (!G::VEC || (M == ROWS_BULK && a.pre_w == nullptr)) {
            if (G::STAGED) g.barrier();
            refill();
        }
        if (a.stats != nullptr && g.tid == 0 && there)
            reinterpret_cast<float4 *>(a.stats)[t] = make_float4(mean0, rstd0, mean1, rstd1);
    }
    g.finish(at, p.stages, a.status);
}

template <typename D, int M, int C> mp_status_t forward(const NormCall &c)
{
    static std::atomic<uint64_t> allowed{0};
    NormArgs a = {};
    a.in.slot[3] = a.in.slot[4] = -1;
    a.in.add(ROW_X, c.x);
    a.in.add(ROW_RESIDUAL, c.residual);
    a.in.add(ROW_GATE, c.gate_rows);
    a.post_w = c.post_w; a.post_b = c.post_b; a.gate = c.gate; a.pre_w = c.pre_w; a.pre_b = c.pre_b;
    a.T = c.T; a.H = c.H; a.kind = c.kind; a.gate_form = c.gate_form; a.eps = c.eps; a.scale = c.scale;
    a.s = c.s_out; a.y = c.y; a.stats = c.stats; a.status = c.status;
    const int held = (c.post_w != nullptr) + (c.post_b != nullptr) + (c.gate_form == MP_GATE_CHANNEL) +
                     (c.pre_w != nullptr) + (c.pre_b != nullptr);
    const NormPlan p = norm_plan<D>(c.T, c.H, C, C < 4 ? NORM_THREADS : 2 * NORM_THREADS, M, a.in.tensors,
                                    held, 0, true);
    if (C < 4 && p.stages < 1) return MP_ERR_UNSUPPORTED;   // there is room for a slot up to 8,192 values of fp32
    int grid;
    return norm_launch(k_block_norm<D, M, C>, allowed, p, M, true, c.T, c.stream, grid, a);
}

}  // namespace

template <typename D> mp_status_t norm_forward(const NormCall &c)
{
    if (c.H > 16 * NORM_THREADS) return c.vec ? forward<D, ROWS_VEC, 4>(c) : forward<D, ROWS_ANY, 4>(c);
    if (!c.vec) return norm_is_narrow(c.H) ? forward<D, ROWS_NARROW, 2>(c) : forward<D, ROWS_ANY, 2>(c);
    return norm_by_bulk<D>(c.H) ? forward<D, ROWS_BULK, 2>(c) : forward<D, ROWS_VEC, 2>(c);
}
template mp_status_t norm_forward<__nv_bfloat16>(const NormCall &);
template mp_status_t norm_forward<__half>(const NormCall &);
template mp_status_t norm_forward<float>(const NormCall &);

}  // namespace mp
