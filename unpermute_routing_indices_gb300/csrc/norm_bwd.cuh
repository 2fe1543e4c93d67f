// Gradients of the norms before and after a block (mp_block_norm_bwd): see norm.cuh for the
// layout and mp.h for the formulas.
//
// One pass over the rows: x, s and the two gradients are read once, g_x, g_residual and
// the gate's gradient written once.  Of what the rows share, a thread sums its columns'
// gradients over its rows in registers (the weights') or in shared memory (biases and a
// gate a channel, for which registers are short); a CTA adds up its groups in order and leaves one
// partial sum a column, and a second kernel adds those of the CTAs in order, in pairs of fp32.  A thread adds up
// T / (152 R) rows one after another (R rows a CTA at a time), a CTA its groups: by the count of roundings off by
// (T / (152 R) + 40) 2^-24 of the sum of magnitudes, 1.5e-5 for 32,768 x 7,168, where a result in bf16 is rounded by 2^-8.
#pragma once

#include "norm.cuh"

namespace mp {
namespace {

enum { SUM_POST_W, SUM_POST_B, SUM_PRE_W, SUM_PRE_B, SUM_GATE };

struct NormBwdArgs {
    NormInputs in;
    const void *post_w, *post_b, *gate, *pre_w;
    const float *stats;
    int64_t T;
    int H, kind, gate_form;
    float scale;
    void *g_x, *g_residual, *g_gate;
    float *sums[NORM_SHARED];
    int32_t *status;
};
enum { ROW_G_S, ROW_G_Y, ROW_S, ROW_X, ROW_GATE };

// MORE: biases, or a gate a channel, whose gradients are summed beside the weights'.  (One kernel for
// both: 621 us in place of 607 for 32,768 x 7,168 without them.)
template <typename D, int M, int C, bool POST, bool PRE, bool MORE>
__global__ void __launch_bounds__(C < 4 ? NORM_THREADS : 2 * NORM_THREADS, 1)
    k_block_norm_bwd(const NormBwdArgs a, const NormPlan p)
{
    typedef NormGroup<D, M, C> G;
    constexpr int N2 = G::N2;
    extern __shared__ __align__(16) uint8_t smem[];
    pdl_trigger();
    pdl_wait();
    G g;
    const int H = a.H;
    g.begin(smem, p.W, p.R, H);
    uint8_t *const rings = smem + G::head(p.W, p.R);
    const int slot_bytes = a.in.tensors * p.pitch;
    uint8_t *const ring = rings + static_cast<size_t>(g.group) * p.stages * slot_bytes;
    // What the rows share, behind the slots.
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
    const D *const post_w = hold(POST ? a.post_w : nullptr), *const pre_w = hold(PRE ? a.pre_w : nullptr);
    const D *const post_b = hold(a.post_b);
    const bool by_channel = a.gate_form == MP_GATE_CHANNEL;
    const D *const channel = hold(by_channel ? a.gate : nullptr);
    // Sums beside the weights', [R] groups each; C 4: the partial sums themselves.
    const int wide = norm_wide(H), pile = N2 * p.W;
    f2 *const more_at = reinterpret_cast<f2 *>(held);
    f2 *more[3];
    {
        constexpr int which[3] = {SUM_POST_B, SUM_PRE_B, SUM_GATE};
        f2 *at = more_at, zero[N2];
#pragma unroll
        for (int i = 0; i < N2; ++i) zero[i] = 0ull;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            more[i] = at + g.group * pile;
            if (!MORE || a.sums[which[i]] == nullptr) continue;
            if constexpr (G::STAGED) {
#pragma unroll
                for (int k = 0; k < N2; ++k) more[i][k * p.W + g.tid] = 0ull;
                at += p.R * pile;
            } else {
                g.template columns<false>(a.sums[which[i]] + static_cast<int64_t>(blockIdx.x) * H, zero);
            }
        }
    }
    const auto add_row = [&](int i, float *sums, const f2 (&v)[N2]) {
        if constexpr (G::STAGED)
            g.pile(more[i], v);
        else
            g.template columns<true>(sums + static_cast<int64_t>(blockIdx.x) * H, v);
    };

    const uint32_t T = static_cast<uint32_t>(a.T), step = gridDim.x * p.R, first = blockIdx.x * p.R;
    cp_commit();
    if (G::STAGED)
        for (int i = 0; i < p.stages; ++i) g.template fetch<1>(a.in, first + i * step + g.group, T, ring + i * slot_bytes, p.pitch, i);

    const bool layer = a.kind == MP_NORM_LAYER, token = a.gate_form == MP_GATE_TOKEN;
    const float inv = 1.0f / static_cast<float>(H);
    f2 post_sum[N2], pre_sum[N2];
#pragma unroll
    for (int i = 0; i < N2; ++i) post_sum[i] = pre_sum[i] = 0ull;

    // What a row has one of, read one row ahead.
    const auto stats_of = [&](uint32_t t) {
        return t < T ? ld_in(reinterpret_cast<const float4 *>(a.stats) + t) : make_float4(0, 0, 0, 0);
    };
    const auto gate_of = [&](uint32_t t) {
        return token && t < T ? norm_value(static_cast<const D *>(a.gate)[t]) : 1.0f;
    };
    float4 next = stats_of(first + g.group);
    float next_gate = gate_of(first + g.group);
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
        const float4 st = next;
        const float gate = next_gate;
        next = stats_of(t + step);
        next_gate = gate_of(t + step);
        g.arrived(at, p.stages, there);
        // Once everyone has read the row, which is so after the last sum that follows the last load,
        // its slot takes the one `stages` steps on.
        bool refilled = false;
        const auto refill = [&]() {
            if (G::STAGED) g.template fetch<1>(a.in, t + p.stages * step, T, slot, p.pitch, at);
            refilled = true;
        };
        const auto load = [&](int which, f2 (&f)[N2]) {
#pragma unroll
            for (int i = 0; i < N2; ++i) f[i] = 0ull;
            if (there && a.in.slot[which] >= 0) g.load(g.row(a.in.rows[which], t, slot + a.in.slot[which] * p.pitch), f);
        };
        // (v - mean) rstd
        const auto standard = [&](f2 (&v)[N2], float mean, float rstd) {
            const f2 off = pair(-mean, -mean), r = pair(rstd, rstd);
            if (layer) {
#pragma unroll
                for (int i = 0; i < N2; ++i) v[i] = add2(v[i], off);
            }
#pragma unroll
            for (int i = 0; i < N2; ++i) v[i] = mul2(v[i], r);
        };
        f2 total[N2];   // the gradient of s
        if (PRE) {
            f2 hat[N2], d[N2];
            load(ROW_S, hat);
            load(ROW_G_Y, d);
            if (MORE && a.sums[SUM_PRE_B] != nullptr && there) add_row(1, a.sums[SUM_PRE_B], d);
            standard(hat, st.z, st.w);
            f2 w[N2];
            g.load_shared(pre_w, w);
            f2 along2 = 0ull, flat2 = 0ull;
#pragma unroll
            for (int i = 0; i < N2; ++i) {   // rows that are not there are 0
                pre_sum[i] = fma2(d[i], hat[i], pre_sum[i]);
                d[i] = mul2(d[i], w[i]);
                along2 = fma2(d[i], hat[i], along2);
            }
            load(ROW_G_S, total);
            float t2[2] = {sum2(along2), 0.0f};
            if (layer) {
#pragma unroll
                for (int i = 0; i < N2; ++i) flat2 = add2(flat2, d[i]);
                t2[1] = sum2(flat2);
                g.sums(t2);
            } else {
                float t1[1] = {t2[0]};
                g.sums(t1);
                t2[0] = t1[0];
            }
            // total = g_s + rstd (d - flat - hat along)
            const float along = -t2[0] * inv, flat = -t2[1] * inv;
            const f2 m = pair(along, along), f = pair(flat, flat), r = pair(st.w, st.w);
            if (!POST && a.gate_form == MP_GATE_NONE) refill();
            if (layer) {
#pragma unroll
                for (int i = 0; i < N2; ++i) d[i] = add2(d[i], f);
            }
#pragma unroll
            for (int i = 0; i < N2; ++i) total[i] = fma2(r, fma2(hat[i], m, d[i]), total[i]);
        } else {
            load(ROW_G_S, total);
        }
        if (a.g_residual != nullptr && there) g.store(static_cast<D *>(a.g_residual) + row, total);
        if (POST || a.gate_form != MP_GATE_NONE || a.scale != 1.0f) {
            const f2 by = pair(a.scale, a.scale);
#pragma unroll
            for (int i = 0; i < N2; ++i) total[i] = mul2(total[i], by);
        }
        if (POST || a.gate_form != MP_GATE_NONE) {
            f2 hat[N2];
            load(ROW_X, hat);
            if (POST) standard(hat, st.x, st.y);
            float t3[3] = {0.0f, 0.0f, 0.0f};
            if (a.gate_form != MP_GATE_NONE) {
                f2 u[N2], k[N2];
                if (POST) {
                    g.load_shared(post_w, k);
#pragma unroll
                    for (int i = 0; i < N2; ++i) u[i] = mul2(hat[i], k[i]);
                    if (a.post_b != nullptr) {
                        g.load_shared(post_b, k);
#pragma unroll
                        for (int i = 0; i < N2; ++i) u[i] = add2(u[i], k[i]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < N2; ++i) u[i] = hat[i];
                }
                f2 gate2 = 0ull;
#pragma unroll
                for (int i = 0; i < N2; ++i) {
                    u[i] = mul2(u[i], total[i]);
                    gate2 = add2(gate2, u[i]);
                }
                t3[2] = sum2(gate2);
                if (MORE && a.sums[SUM_GATE] != nullptr && there) add_row(2, a.sums[SUM_GATE], u);
                // The gate is read before its gradient is written, which may take its place.
                if (token) {
#pragma unroll
                    for (int i = 0; i < N2; ++i) k[i] = pair(gate, gate);
                } else if (by_channel) {
                    g.load_shared(channel, k);
                } else {
                    load(ROW_GATE, k);
                }
                if (a.gate_form == MP_GATE_ELEMENT && a.g_gate != nullptr && there)
                    g.store(static_cast<D *>(a.g_gate) + row, u);
#pragma unroll
                for (int i = 0; i < N2; ++i) total[i] = mul2(total[i], k[i]);
            }
            if (POST) {
                if (MORE && a.sums[SUM_POST_B] != nullptr && there) add_row(0, a.sums[SUM_POST_B], total);
                asm volatile("" ::: "memory");   // the weights are read again: registers are short
                f2 along2 = 0ull, flat2 = 0ull, w[N2];
                g.load_shared(post_w, w);
#pragma unroll
                for (int i = 0; i < N2; ++i) {
                    post_sum[i] = fma2(total[i], hat[i], post_sum[i]);
                    total[i] = mul2(total[i], w[i]);
                    along2 = fma2(total[i], hat[i], along2);
                    flat2 = add2(flat2, total[i]);
                }
                t3[0] = sum2(along2);
                t3[1] = sum2(flat2);
            }
            if (layer || token) {
                g.sums(t3);
            } else if (POST) {
                float t1[1] = {t3[0]};
                g.sums(t1);
                t3[0] = t1[0];
            }
            if (POST || layer || token) refill();
            if (token && a.g_gate != nullptr && g.tid == 0 && there) norm_put(static_cast<D *>(a.g_gate) + t, t3[2]);
            if (POST) {
                const float along = -t3[0] * inv, flat = layer ? -t3[1] * inv : 0.0f;
                const f2 m = pair(along, along), f = pair(flat, flat), r = pair(st.y, st.y);
                if (layer) {
#pragma unroll
                    for (int i = 0; i < N2; ++i) total[i] = add2(total[i], f);
                }
#pragma unroll
                for (int i = 0; i < N2; ++i) total[i] = mul2(r, fma2(hat[i], m, total[i]));
            }
        }
        if (a.g_x != nullptr && there) g.store(static_cast<D *>(a.g_x) + row, total);
        if (!refilled) {
            if (G::STAGED) g.barrier();
            refill();
        }
        at = g.after(at, p.stages);
    }
    g.finish(at, p.stages, a.status);

    // The groups' sums, in their order, into this CTA's partial sums.  The slots are free now.
    float *const stack = reinterpret_cast<float *>(rings);
    const int low = threadIdx.x & 31;
    const int piles = p.W < 32 ? (p.W * p.R + 31) / 32 : p.R, own = p.W < 32 ? threadIdx.x >> 5 : g.group;
    const auto pile_up = [&](float *sums, f2 (&v)[N2]) {
        if (sums == nullptr) return;
        float *const to = sums + static_cast<int64_t>(blockIdx.x) * H;
        if (!G::STAGED) {
            g.template columns<false>(to, v);
            return;
        }
        __syncthreads();
        for (int d = p.W; d < 32; d *= 2)
#pragma unroll
            for (int i = 0; i < N2; ++i) v[i] = add2(v[i], __shfl_xor_sync(FULL_MASK, v[i], d));
        if (p.W >= 32 || low < p.W) g.template columns<false>(stack + own * wide, v);
        __syncthreads();
        for (int c = threadIdx.x; c < H; c += blockDim.x) {
            float s = 0.0f;
            for (int i = 0; i < piles; ++i) s += stack[i * wide + c];
            to[c] = s;
        }
    };
    if (POST) pile_up(a.sums[SUM_POST_W], post_sum);
    if (PRE) pile_up(a.sums[SUM_PRE_W], pre_sum);
    if constexpr (MORE && G::STAGED) {
        const f2 *from = more_at;
        __syncthreads();
        for (const int k : {SUM_POST_B, SUM_PRE_B, SUM_GATE}) {
            if (a.sums[k] == nullptr) continue;
            float *const to = a.sums[k] + static_cast<int64_t>(blockIdx.x) * H;
            for (int c = threadIdx.x; c < H; c += blockDim.x) {
                float s = 0.0f;
                for (int i = 0; i < p.R; ++i) s += g.piled(from + i * pile, c);
                to[c] = s;
            }
            from += p.R * pile;
        }
    }
}

template <typename D, int M, int C, bool POST, bool PRE, bool MORE> mp_status_t launch(const NormCall &c, const NormBwdArgs &a,
                                                                                         const NormPlan &p, int &parts)
{
    static std::atomic<uint64_t> allowed{0};
    return norm_launch(k_block_norm_bwd<D, M, C, POST, PRE, MORE>, allowed, p, M, false, c.T, c.stream, parts, a);
}

template <typename D, int M, int C, bool POST, bool PRE> mp_status_t run(const NormCall &c, int &parts)
{
    NormBwdArgs a = {};
    a.in.add(ROW_G_S, c.g_s);
    a.in.add(ROW_G_Y, c.g_y);
    a.in.add(ROW_S, c.s);
    a.in.add(ROW_X, POST || c.gate_form != MP_GATE_NONE ? c.x : NormRows{});
    a.in.add(ROW_GATE, c.gate_rows);
    a.post_w = c.post_w; a.post_b = c.post_b; a.gate = c.gate; a.pre_w = c.pre_w;
    a.stats = c.stats; a.T = c.T; a.H = c.H; a.kind = c.kind; a.gate_form = c.gate_form; a.scale = c.scale;
    a.g_x = c.g_x; a.g_residual = c.g_residual; a.g_gate = c.g_gate; a.status = c.status;
    for (int i = 0; i < NORM_SHARED; ++i) a.sums[i] = c.sums[i];
    const int more = (c.sums[SUM_POST_B] != nullptr) + (c.sums[SUM_PRE_B] != nullptr) + (c.sums[SUM_GATE] != nullptr);
    const int held = POST + PRE + (c.post_b != nullptr) + (c.gate_form == MP_GATE_CHANNEL);
    const NormPlan p = norm_plan<D>(c.T, c.H, C, C < 4 ? NORM_THREADS : 2 * NORM_THREADS, M, a.in.tensors,
                                    held, more, false);
    if constexpr (C < 4) {
        if (p.stages < 1)   // one fp32 row and the sums beside it are more than shared memory: 5,121 wide or more
            return run<D, NormGroup<D, M, C>::VEC ? ROWS_VEC : ROWS_ANY, 4, POST, PRE>(c, parts);
        if (more == 0) return launch<D, M, C, POST, PRE, false>(c, a, p, parts);
    }
    return launch<D, M, C, POST, PRE, true>(c, a, p, parts);
}

template <typename D, int M, int C> mp_status_t by_norms(const NormCall &c, int &parts)
{
    if (c.post_w == nullptr) return run<D, M, C, false, true>(c, parts);
    return c.pre_w == nullptr ? run<D, M, C, true, false>(c, parts) : run<D, M, C, true, true>(c, parts);
}

}  // namespace

template <typename D> mp_status_t norm_backward(const NormCall &c, int &parts)
{
    if (c.H > 16 * NORM_THREADS) return c.vec ? by_norms<D, ROWS_VEC, 4>(c, parts) : by_norms<D, ROWS_ANY, 4>(c, parts);
    if (!c.vec) return norm_is_narrow(c.H) ? by_norms<D, ROWS_NARROW, 2>(c, parts) : by_norms<D, ROWS_ANY, 2>(c, parts);
    return norm_by_bulk<D>(c.H) ? by_norms<D, ROWS_BULK, 2>(c, parts) : by_norms<D, ROWS_VEC, 2>(c, parts);
}

}  // namespace mp
