// The whole mixture-of-experts layer for a few tokens.
//
//   l = x router^T;  (idx, w) = the router's choice;
//   y[t] = sum_k w[t,k] (act(x[t] w1[e]^T + b1[e]) w2[e]^T + b2[e]),  e = idx[t,k]
//
// The picked experts' weights are read once and bound it; rows are nothing beside them.  Two
// kernels: k_layer_logits, a CTA for each expert, and k_layer, which runs from the choice to the
// result on every SM.  One token's choice every CTA makes for itself; several tokens' are
// spread over the CTAs, and the grid waits for them.
//
// Logits are sums in pairs of fp32 (a sum and what its roundings lost), so that they are those
// of 64 bits rounded once, and the choice with them.  (FP64 units are few on this part: 1.25
// TFLOP/s by its data sheet.)
//
// k_layer: one CTA an SM, launched cooperatively.  A unit of work is U rows of an expert's
// weights against all tokens of that expert (an entry: up to 8 NT of them).  Each of eight
// warps multiplies 16 weight rows by its share of the columns, 128 a stage, which it copies
// itself, by cp.async into a ring of its own; one more warp copies the tokens' rows for all, two
// join the eight warps' sums, in a fixed order, and apply bias and activation, so that the
// eight never wait for a unit's end, and one claims the units, in order and a little ahead, since
// SMs do not get equal shares of the memory (an equal share of units each: 10% at 64 tokens).
// (mma.m16n8k16: weight rows are its 16, tokens its 8.  Bytes bound it, so the tensor cores'
// older form is enough, and it needs no tile of 128 rows.)  The rings do not stop between the
// two products: the second's units of an expert need the activations h of that expert alone, and
// a count for each expert's entry says when they are there, long before its turn; with a barrier
// of the grid instead, the SMs stood idle for 6 us (one token) to 12 us (64).  h is kept as two bf16 values, the
// nearest one and the nearest of what is left, 16 bits of it in all: the second product takes
// both, which costs no time, and y's error is that of its own rounding (with one: 1.4 times that).
// Sums over an expert's rows stay in fp32 until every slot of a token is there; a second
// barrier, and the slots are added in order.
// (Weights by bulk copies of row pieces, one warp for all: 2 KB pieces 56 us for one token of
// 128 experts of 1,024 x 4,096, 512-byte pieces 393 us for 64 tokens of 64 of 1,024 x 2,048.)
//
// A stage of a warp is 16 rows of 256 bytes; the rows' 64-byte halves are swapped in every
// other row, so that the 16-byte reads of eight lanes (two rows, four pieces) touch all banks
// once.  Lane (g, c) reads columns 8c .. 8c+7 of 32 in one load and feeds them to two products
// as if they were the fragment's k = 2c, 2c+1, 2c+8, 2c+9: both operands agree on that order,
// which is all that a sum over k asks.
#include "expert.cuh"
#include "pairs.cuh"
#include "route.cuh"
#include "tc.cuh"

#include <type_traits>

namespace mp {
namespace {

constexpr int LOGIT_THREADS = 128, LOGIT_WARPS = LOGIT_THREADS / 32;
constexpr int MATH_WARPS = 8, MATH_THREADS = 32 * MATH_WARPS;
constexpr int COPY_WARP = MATH_WARPS, CLAIM_WARP = MATH_WARPS + 1, JOIN_WARPS = 2, JOIN_THREADS = 32 * JOIN_WARPS;
constexpr int LAYER_THREADS = MATH_THREADS + 64 + JOIN_THREADS;   // 12 warps: 168 registers a thread
constexpr int CLAIMS = 16, CLAIM_AHEAD = 2;   // units known to a CTA at most; beyond the one whose copies start
constexpr int STAGE_COLS = 128;          // of a warp
constexpr int ROW_PAD = 64;              // bytes between tokens' rows
constexpr int B_MOST = 8, RED_MOST = 4;  // slots for tokens' rows, buffers of sums
constexpr size_t LAYER_SMEM = 227 * 1024;

struct LayerControl {
    unsigned arrived[2];   // CTAs at the barriers of k_layer: after the choice, after the products
    unsigned claimed;      // units
    unsigned done[MP_MAX_EXPERTS + MP_MAX_LAYER_TOKENS * 32 / 8];   // units of the first product, by entry
};

struct LayerArgs {
    const mp_bf16_t *x, *w1, *b1, *w2, *b2;
    const void *router;
    RouteArgs route;
    int T, E, K, H, F, O, act;
    int32_t *idx;
    float *weights;
    mp_bf16_t *y;
    int32_t *status;
    // workspace
    LayerControl *control;
    float *logits;          // [T,E]
    mp_bf16_t *xp;          // [T,Hp]: x with rows of whole 16 bytes, NULL where x is that
    mp_bf16_t *h;           // [T*K,2,Fp]: nearest values, and the nearest of what is left
    float *out;             // [T*K,O]: each slot's result
    int Hp, Fp;
};

__device__ __forceinline__ float bf16_value(const mp_bf16_t *p)
{
    return __uint_as_float(static_cast<uint32_t>(ld_in(p)) << 16);
}

// ---------------------------------------------------------------------------
// logits
// ---------------------------------------------------------------------------

// Sums of fp32 values and what their roundings lost (Knuth's two-sum), two side by side.
struct PairSums {
    f2 s = 0ull, lost = 0ull;
    __device__ __forceinline__ void add(f2 p)
    {
        const f2 minus = pair(-1.0f, -1.0f);
        const f2 t = add2(s, p), z = fma2(s, minus, t);   // t - s, rounded once
        lost = add2(lost, add2(fma2(fma2(z, minus, t), minus, s), fma2(z, minus, p)));
        s = t;
    }
    // a b, and what the product's rounding lost (nothing for two bf16 values)
    template <bool EXACT> __device__ __forceinline__ void add_product(f2 a, f2 b)
    {
        const f2 p = mul2(a, b);
        if (!EXACT) lost = add2(lost, fma2(a, b, mul2(p, pair(-1.0f, -1.0f))));
        add(p);
    }
    __device__ __forceinline__ void add(const PairSums &o)
    {
        add(o.s);
        lost = add2(lost, o.lost);
    }
    // The sum of both.
    __device__ __forceinline__ float total() const
    {
        const float2 v = both(s), l = both(lost);
        const float t = __fadd_rn(v.x, v.y), z = __fsub_rn(t, v.x);
        const float rest = __fadd_rn(__fadd_rn(l.x, l.y), __fadd_rn(__fsub_rn(v.x, __fsub_rn(t, z)), __fsub_rn(v.y, z)));
        return isfinite(t) ? __fadd_rn(t, rest) : t;
    }
};

// Logits of one expert and TB tokens, a CTA each; the first CTAs also clear k_layer's counts and
// lay x out in rows of whole 16 bytes where k_layer wants that.  VEC: rows of x and the
// router are whole chunks of 4 on 16 (8) bytes.
template <typename L, int TB, bool VEC> __global__ void __launch_bounds__(LOGIT_THREADS) k_layer_logits(const LayerArgs a)
{
    __shared__ PairSums part[LOGIT_WARPS][TB];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = blockIdx.x, t0 = blockIdx.y * TB;
    if (e == 0 && t0 == 0)
        for (int i = threadIdx.x; i < static_cast<int>(sizeof(LayerControl) / 4); i += LOGIT_THREADS)
            reinterpret_cast<unsigned *>(a.control)[i] = 0;
    if (a.xp != nullptr)
        for (int t = t0 + e; t < min(t0 + TB, a.T); t += gridDim.x)
            for (int c = threadIdx.x; c < a.Hp; c += LOGIT_THREADS)
                a.xp[static_cast<int64_t>(t) * a.Hp + c] = c < a.H ? a.x[static_cast<int64_t>(t) * a.H + c] : 0;
    const mp_bf16_t *x[TB];
#pragma unroll
    for (int b = 0; b < TB; ++b) x[b] = a.x + static_cast<int64_t>(min(t0 + b, a.T - 1)) * a.H;
    const L *r = static_cast<const L *>(a.router) + static_cast<int64_t>(e) * a.H;
    PairSums v[TB];
    if (VEC) {
        typedef typename std::conditional<sizeof(L) == 4, float4, uint2>::type Four;
#pragma unroll(TB == 1 ? 8 : 4)
        for (int c = threadIdx.x * 4; c < a.H; c += LOGIT_THREADS * 4) {
            const Four w = ld_in(reinterpret_cast<const Four *>(r + c));
            const L *wl = reinterpret_cast<const L *>(&w);
            const f2 w0 = pair(logit_value(wl[0]), logit_value(wl[1])), w1 = pair(logit_value(wl[2]), logit_value(wl[3]));
#pragma unroll
            for (int b = 0; b < TB; ++b) {
                const uint2 u = ld_in(reinterpret_cast<const uint2 *>(x[b] + c));
                v[b].template add_product<sizeof(L) == 2>(pair(bf16_lo(u.x), bf16_hi(u.x)), w0);
                v[b].template add_product<sizeof(L) == 2>(pair(bf16_lo(u.y), bf16_hi(u.y)), w1);
            }
        }
    } else {
#pragma unroll 4
        for (int c = threadIdx.x; c < a.H; c += LOGIT_THREADS) {
            const f2 w = pair(logit(r + c), 0.0f);
#pragma unroll
            for (int b = 0; b < TB; ++b) v[b].template add_product<sizeof(L) == 2>(pair(bf16_value(x[b] + c), 0.0f), w);
        }
    }
#pragma unroll
    for (int b = 0; b < TB; ++b) {
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            PairSums o;
            o.s = __shfl_xor_sync(FULL_MASK, v[b].s, d);
            o.lost = __shfl_xor_sync(FULL_MASK, v[b].lost, d);
            v[b].add(o);
        }
        if (lane == 0) part[warp][b] = v[b];
    }
    __syncthreads();
    if (threadIdx.x < TB && t0 + static_cast<int>(threadIdx.x) < a.T) {
        PairSums s = part[0][threadIdx.x];
        for (int w = 1; w < LOGIT_WARPS; ++w) s.add(part[w][threadIdx.x]);
        a.logits[static_cast<int64_t>(t0 + threadIdx.x) * a.E + e] = s.total();
    }
}

// ---------------------------------------------------------------------------
// from the choice to the result
// ---------------------------------------------------------------------------

// Weights are read once: they leave L2 before anything else does.
__device__ __forceinline__ uint64_t read_once()
{
    uint64_t policy;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    return policy;
}
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, uint64_t policy, int bytes = 16)
{
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(bytes),
                 "l"(policy)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but this thread's last S groups of copies have landed.
template <int S> __device__ __forceinline__ void copy_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(S) : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async;" ::: "memory"); }
__device__ __forceinline__ uint4 lds128(uint32_t at)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t at)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at));
    return v;
}
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// A wait whose end the whole warp agrees on.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *gave_up)
{
    return __all_sync(FULL_MASK, mbar_wait(bar, parity, gave_up)) != 0;
}
// The joining warps; they and the multiplying ones.  A warp comes to a barrier as a whole.
__device__ __forceinline__ void join_barrier()
{
    __syncwarp();
    asm volatile("bar.sync 1, %0;" ::"n"(JOIN_THREADS) : "memory");
}
// Whether all of the joining threads say so; a barrier of them too.
__device__ __forceinline__ bool join_all(bool v)
{
    uint32_t all;
    __syncwarp();
    asm volatile("{\n\t.reg .pred p, q;\n\t"
                 "setp.ne.u32 q, %1, 0;\n\t"
                 "bar.red.and.pred p, 1, %2, q;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(all)
                 : "r"(static_cast<uint32_t>(v)), "n"(JOIN_THREADS)
                 : "memory");
    return all != 0;
}
__device__ __forceinline__ void most_barrier()
{
    __syncwarp();
    asm volatile("bar.sync 2, %0;" ::"n"(MATH_THREADS + JOIN_THREADS) : "memory");
}

// Waits until there have been `count` arrivals; at most 4 s.
__device__ __forceinline__ bool grid_wait(const unsigned *arrived, unsigned count, volatile int *gave_up)
{
    const uint64_t t0 = now_ns();
    for (int i = 0;; ++i) {
        unsigned n;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(n) : "l"(arrived) : "memory");
        if (n >= count) return true;
        if (*gave_up) return false;
        if ((i & 63) == 63 && now_ns() - t0 > WAIT_NS) {
            *gave_up = 1;
            return false;
        }
    }
}
__device__ __forceinline__ void grid_arrive(unsigned *arrived)
{
    asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(arrived) : "memory");
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

// One token's choice by one warp.
__device__ __noinline__ void route_one(const RouteArgs &r, const float *logits, int t, int lane)
{
    if (r.E <= 128 && r.K == 8)
        route_token<float, 4, 8>(r, logits, t, lane);
    else if (r.E <= 128)
        route_token<float, 4, 0>(r, logits, t, lane);
    else if (r.E <= 256)
        route_token<float, 8, 0>(r, logits, t, lane);
    else
        route_token<float, 32, 0>(r, logits, t, lane);
}

// How a product is cut.  The eight warps are RG groups of 16 weight rows by KG shares of a stage's
// columns, RG KG = 8: a unit is U = 16 RG rows, a stage KC = 128 KG columns.
struct Cut {
    int log_kg;
    int b_stages;   // slots for the tokens' rows
    __host__ __device__ int kg() const { return 1 << log_kg; }
    __host__ __device__ int u() const { return 128 >> log_kg; }
    __host__ __device__ int kc() const { return STAGE_COLS << log_kg; }
    __host__ __device__ int b_pitch() const { return kc() * 2 + ROW_PAD; }
};
struct LayerCuts {
    Cut of[2];      // of the first product and of the second
    int b_rows;     // tokens' rows in a slot; twice as many of the second product, both values of h
    int b_second;   // bytes from the first product's slots to the second's
    int reds;       // buffers for the units' sums
};

// Up to 8 NT tokens an entry.  ODD: weight rows that start anywhere.
template <int NT, bool ODD> struct Layer {
    static constexpr int TOKENS = 8 * NT;
    static constexpr int W_PITCH = STAGE_COLS * 2 + (ODD ? 16 : 0);   // a row that starts anywhere takes a granule more
    static constexpr int W_STAGE = MATH_WARPS * 16 * W_PITCH;
    static constexpr int STAGES = NT == 4 ? 3 : 4;
    static constexpr int RED = 160 * TOKENS;   // floats: KG columns' shares, TOKENS, U rows and 4 to part the banks
    struct Entry {
        int expert, first, count;   // tokens' routes: order[first ..]
    };
    struct Unit {
        int p, entry, block;   // product (2: no more units), entry, rows
    };
    struct Shared {
        uint64_t b_full[2][B_MOST], b_empty[2][B_MOST], red_full[RED_MOST], red_empty[RED_MOST];
        uint64_t claim_full[CLAIMS], claim_seen[CLAIMS], claim_empty[CLAIMS];
        Unit unit[CLAIMS];
        int32_t idx[32];      // of one token
        float weights[32];
        int gave_up, entries;
    };
    // After the rings: what is above, the units' sums, and the routes: tokens of each expert (a bit
    // each), where an expert's routes start, routes by expert, entries.
    static constexpr size_t tables(int E, int R)
    {
        return sizeof(Shared) + (3 * static_cast<size_t>(E) + R) * 4 + ((E < R ? E : R) + R / TOKENS) * sizeof(Entry) + 16;
    }
};

template <int NT, bool ODD>
__global__ void __launch_bounds__(LAYER_THREADS, 1) k_layer(const LayerArgs a, const LayerCuts cuts, const int b_bytes)
{
    typedef Layer<NT, ODD> L;
    constexpr int TOKENS = L::TOKENS, STAGES = L::STAGES, CHAINS = NT == 1 ? 4 : 2;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, R = a.T * a.K;
    const uint32_t b_ring = smem_u32(smem) + STAGES * L::W_STAGE;
    uint8_t *at = smem + STAGES * L::W_STAGE + b_bytes;
    typename L::Shared &s = *reinterpret_cast<typename L::Shared *>(at);
    at += sizeof(typename L::Shared);
    float *const red = reinterpret_cast<float *>(at);
    at += cuts.reds * L::RED * 4;
    unsigned *const tokens_of = reinterpret_cast<unsigned *>(at);
    int *const start = reinterpret_cast<int *>(tokens_of + 2 * a.E), *const order = start + a.E;
    typename L::Entry *const entry = reinterpret_cast<typename L::Entry *>(order + R);
    volatile int *gave_up = &s.gave_up;

    if (threadIdx.x == 0) {
        for (int p = 0; p < 2; ++p)
            for (int i = 0; i < B_MOST; ++i) {
                mbar_init(smem_u32(&s.b_full[p][i]), 1);
                mbar_init(smem_u32(&s.b_empty[p][i]), MATH_WARPS);
            }
        for (int i = 0; i < RED_MOST; ++i) {
            mbar_init(smem_u32(&s.red_full[i]), MATH_WARPS);
            mbar_init(smem_u32(&s.red_empty[i]), JOIN_WARPS);
        }
        for (int i = 0; i < CLAIMS; ++i) {
            mbar_init(smem_u32(&s.claim_full[i]), 1);
            mbar_init(smem_u32(&s.claim_seen[i]), MATH_WARPS);
            mbar_init(smem_u32(&s.claim_empty[i]), MATH_WARPS + 1 + JOIN_WARPS);
        }
        mbar_init_fence();
        s.gave_up = 0;
    }
    for (int e = threadIdx.x; e < 2 * a.E; e += LAYER_THREADS) tokens_of[e] = 0;
    pdl_trigger();
    pdl_wait();
    __syncthreads();

    const int32_t *idx = a.idx;
    const float *weights = a.weights;
    if (a.T == 1) {
        if (warp == 0) {
            RouteArgs r = a.route;
            r.idx = s.idx;
            r.weights = s.weights;
            route_one(r, a.logits, 0, lane);
            __syncwarp();
            if (blockIdx.x == 0 && lane < a.K) {
                a.idx[lane] = s.idx[lane];
                a.weights[lane] = s.weights[lane];
            }
        }
        idx = s.idx;
        weights = s.weights;
        __syncthreads();
    } else {
        if (warp == 0) {
            for (int t = blockIdx.x; t < a.T; t += gridDim.x) route_one(a.route, a.logits + static_cast<int64_t>(t) * a.E, t, lane);
            __threadfence();
            __syncwarp();
            if (lane == 0) {
                grid_arrive(&a.control->arrived[0]);
                (void)grid_wait(&a.control->arrived[0], gridDim.x, gave_up);
            }
        }
        __syncthreads();
    }
    // The routes of each expert in the tokens' order (every CTA has to come to the same entries), and
    // entries of up to TOKENS of them.  After a wait given up idx may be anything: there are none.
    const int routes_there = *gave_up ? 0 : R;
    for (int r = threadIdx.x; r < routes_there; r += LAYER_THREADS) {
        const int e = idx[r], t = r / a.K;
        if (e >= 0) atomicOr(tokens_of + 2 * e + (t >> 5), 1u << (t & 31));
    }
    __syncthreads();
    if (warp == 0) {
        // Each lane takes a run of experts, so that the sums cross the warp once.
        const int run = (a.E + 31) / 32, e0 = min(lane * run, a.E), e1 = min(e0 + run, a.E);
        const auto routes_of = [&](int e) { return __popc(tokens_of[2 * e]) + __popc(tokens_of[2 * e + 1]); };
        int routes = 0, entries = 0;
        for (int e = e0; e < e1; ++e) {
            const int n = routes_of(e);
            routes += n;
            entries += (n + TOKENS - 1) / TOKENS;
        }
        int first = routes, slot = entries;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(FULL_MASK, first, d), q = __shfl_up_sync(FULL_MASK, slot, d);
            if (lane >= d) {
                first += o;
                slot += q;
            }
        }
        if (lane == 31) s.entries = slot;
        first -= routes;
        slot -= entries;
        for (int e = e0; e < e1; ++e) {
            const int n = routes_of(e);
            start[e] = first;
            for (int i = 0; i < n; i += TOKENS) entry[slot++] = {e, first + i, min(TOKENS, n - i)};
            first += n;
        }
    }
    __syncthreads();
    for (int r = threadIdx.x; r < routes_there; r += LAYER_THREADS) {
        const int e = idx[r], t = r / a.K;
        if (e < 0) continue;
        const unsigned low = tokens_of[2 * e], high = tokens_of[2 * e + 1], below = (1u << (t & 31)) - 1u;
        order[start[e] + (t < 32 ? __popc(low & below) : __popc(low) + __popc(high & below))] = r;
    }
    __syncthreads();

    const bool gated = act_gated(a.act);
    const int entries = s.entries;
    const int FU = gated ? cuts.of[0].u() / 2 : cuts.of[0].u();   // columns of h that a unit makes
    const int blocks0 = (a.F + FU - 1) / FU, blocks1 = (a.O + cuts.of[1].u() - 1) / cuts.of[1].u();
    const int rows_of[2] = {a.F * (gated ? 2 : 1), a.O};   // of one expert
    // Unit i of this CTA, once it is claimed.
    const auto unit_at = [&](int i, typename L::Unit &u) {
        const bool there = warp_wait(smem_u32(&s.claim_full[i % CLAIMS]), (i / CLAIMS) & 1, gave_up);
        if (there) u = s.unit[i % CLAIMS];
        return there && u.p < 2;
    };
    const auto unit_done = [&](int i) {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s.claim_empty[i % CLAIMS]));
    };

    if (warp == CLAIM_WARP) {
        // Units of the first product come before all of the second: those wait for them.
        if (lane != 0) return;
        const int first = entries * blocks0, all = first + entries * blocks1;
        for (int i = 0;; ++i) {
            if (i > CLAIM_AHEAD) {
                const int seen = i - 1 - CLAIM_AHEAD;
                if (!mbar_wait(smem_u32(&s.claim_seen[seen % CLAIMS]), (seen / CLAIMS) & 1, gave_up)) return;
            }
            if (!mbar_wait(smem_u32(&s.claim_empty[i % CLAIMS]), ((i / CLAIMS) & 1) ^ 1, gave_up)) return;
            const int u = static_cast<int>(atomicAdd(&a.control->claimed, 1u));
            const int p = u >= first, at = p ? u - first : u, nb = p ? blocks1 : blocks0;
            typename L::Unit &to = s.unit[i % CLAIMS];
            to.entry = at / nb;
            to.block = at - to.entry * nb;
            to.p = u < all ? p : 2;
            mbar_arrive(smem_u32(&s.claim_full[i % CLAIMS]));
            if (u >= all) return;
        }
    }
    if (warp == COPY_WARP) {
        // The tokens' rows: x, then h.
        int at_stage[2] = {0, 0}, issued[2] = {0, 0}, there = -1;   // there: the last entry whose h is
        uint32_t phase[2] = {0, 0};
        bool on = true;
        typename L::Unit u;
        for (int i = 0; on && unit_at(i, u); ++i) {
            const int p = u.p, K = p == 0 ? a.Hp : a.Fp, KC = cuts.of[p].kc();
            const int pitch = cuts.of[p].b_pitch(), slot = cuts.b_rows * (p + 1) * pitch;
            const uint32_t ring = b_ring + (p == 0 ? 0 : cuts.b_second);
            const typename L::Entry en = entry[u.entry];
            if (p == 1 && u.entry != there) {
                there = u.entry;
                if (lane == 0) on = grid_wait(&a.control->done[there], blocks0, gave_up);
                on = __shfl_sync(FULL_MASK, static_cast<int>(on), 0) != 0;
                if (!on) break;
                __syncwarp();
                fence_async();   // what other SMs stored, by the copies to come
            }
            const mp_bf16_t *row = p == 0 ? (a.xp != nullptr ? a.xp : a.x) : a.h;
            if (lane < en.count) {
                const int r = order[en.first + lane];
                row += static_cast<int64_t>(p == 0 ? r / a.K : 2 * r) * K;
            }
            int st = at_stage[p], n = issued[p];
            uint32_t ph = phase[p];
            for (int k0 = 0; k0 < K; k0 += KC) {
                on = warp_wait(smem_u32(&s.b_empty[p][st]), ph ^ 1u, gave_up);
                if (!on) break;
                const uint32_t bar = smem_u32(&s.b_full[p][st]), to = ring + st * slot;
                const uint32_t bytes = static_cast<uint32_t>(min(KC, K - k0)) * 2u;
                if (lane == 0) mbar_expect(bar, bytes * en.count * (p + 1));
                __syncwarp();
                if (lane < en.count) {
                    bulk_load(to + lane * pitch, row + k0, bytes, bar);
                    if (p == 1) bulk_load(to + (cuts.b_rows + lane) * pitch, row + K + k0, bytes, bar);
                }
                if (n < B_MOST) ++n;
                if (++st == cuts.of[p].b_stages) {
                    st = 0;
                    ph ^= 1u;
                }
            }
            at_stage[p] = st; issued[p] = n; phase[p] = ph;
            unit_done(i);
        }
        if (*gave_up && lane == 0)   // copies in flight land before the shared memory goes
            for (int p = 0; p < 2; ++p)
                for (int i = 0; i < cuts.of[p].b_stages && i < issued[p]; ++i) {
                    if (--at_stage[p] < 0) {
                        at_stage[p] = cuts.of[p].b_stages - 1;
                        phase[p] ^= 1u;
                    }
                    mbar_drain(smem_u32(&s.b_full[p][at_stage[p]]), phase[p]);
                }
        return;
    }
    if (warp < MATH_WARPS) {
        const int g = lane >> 2, c = lane & 3;
        uint8_t *const ring = smem + warp * 16 * L::W_PITCH;
        const uint64_t policy = read_once();
        // Rows of a group of 16, as they lie in the expert's weights: 8 from `first` on, and 8 from
        // first + 8 + jump on, of which some are there.
        struct Rows {
            int first, jump, there[2];
        };
        const auto rows_at = [&](int p, int block, int rg) {
            Rows r;
            if (p == 0 && gated) {   // 8 of the gate, 8 of the other half
                r.first = block * FU + rg * 8;
                r.jump = a.F - 8;
                r.there[0] = r.there[1] = a.F - r.first;
            } else {
                r.first = block * cuts.of[p].u() + rg * 16;
                r.jump = 0;
                r.there[0] = (p == 0 ? a.F : a.O) - r.first;
                r.there[1] = r.there[0] - 8;
            }
            return r;
        };
        // The stage that is copied next.
        int f_i = 0, f_p = 0, f_k = 0, f_depth = 0, f_col = 0;   // unit, product, first column, all columns, this warp's first
        const char *f_row = nullptr;   // the first row, at this warp's columns
        int64_t f_jump = 0;
        unsigned f_rows = 0;           // a bit for each of the 16 rows that is there
        const auto aim = [&]() {
            typename L::Unit u;
            if (!unit_at(f_i, u)) {
                f_p = 2;
                return;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&s.claim_seen[f_i % CLAIMS]));
            ++f_i;
            f_p = u.p;
            f_k = 0;
            f_depth = f_p == 0 ? a.H : a.F;
            f_col = (warp & (cuts.of[f_p].kg() - 1)) * STAGE_COLS;
            const Rows r = rows_at(f_p, u.block, warp >> cuts.of[f_p].log_kg);
            f_row = reinterpret_cast<const char *>(f_p == 0 ? a.w1 : a.w2) +
                    ((static_cast<int64_t>(entry[u.entry].expert) * (f_p == 0 ? rows_of[0] : rows_of[1]) + r.first) * f_depth + f_col) * 2;
            f_jump = static_cast<int64_t>(r.jump) * f_depth * 2;
            f_rows = ((1u << min(max(r.there[0], 0), 8)) - 1u) | ((1u << min(max(r.there[1], 0), 8)) - 1u) << 8;
        };
        const auto fetch = [&](int stage) {
            if (f_p < 2) {
                const int n = f_depth - f_k - f_col;   // columns that are there
                const uint32_t to = smem_u32(ring + stage * L::W_STAGE);
                if (!ODD) {
                    // A lane: 16 bytes of each other row.
                    const int piece = lane & 15, row = lane >> 4;
                    if (piece * 8 < n) {
                        const uint32_t dst = to + row * L::W_PITCH + (piece ^ row << 2) * 16;
                        const char *const src = f_row + f_k * 2 + piece * 16 + static_cast<int64_t>(row) * 2 * f_depth;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (f_rows >> (row + 2 * i) & 1)
                                copy16(dst + 2 * i * L::W_PITCH, src + static_cast<int64_t>(i) * 4 * f_depth + (i >= 4 ? f_jump : 0), policy);
                    }
                } else if (n > 0) {
                    // The granules of 16 bytes, up to 17 a row, that hold the piece; of the tensor's first
                    // and last, which may reach beyond it, only what is of it is read.
                    const char *const base = reinterpret_cast<const char *>(f_p == 0 ? a.w1 : a.w2);
                    const char *const end = base + static_cast<int64_t>(f_p == 0 ? rows_of[0] : rows_of[1]) * a.E * f_depth * 2;
                    const int bytes = min(n, STAGE_COLS) * 2;
#pragma unroll
                    for (int i = 0; i < 9; ++i) {
                        const int j = lane + 32 * i, row = j / 17, gran = j - 17 * row;
                        if (j >= 16 * 17 || !(f_rows >> row & 1)) continue;
                        const char *const first = f_row + f_k * 2 + static_cast<int64_t>(row) * 2 * f_depth + (row >= 8 ? f_jump : 0);
                        const char *const src = reinterpret_cast<const char *>(reinterpret_cast<uintptr_t>(first) & ~static_cast<uintptr_t>(15)) + gran * 16;
                        if (src >= first + bytes) continue;
                        const uint32_t dst = to + row * L::W_PITCH + gran * 16;
                        if (src >= base) {
                            copy16(dst, src, policy, end - src < 16 ? static_cast<int>(end - src) : 16);
                        } else {
                            for (const char *v = first; v < src + 16 && v < first + bytes; v += 2)
                                asm volatile("st.shared.u16 [%0], %1;" ::"r"(dst + static_cast<uint32_t>(v - src)),
                                             "h"(ld_in(reinterpret_cast<const uint16_t *>(v))) : "memory");
                        }
                    }
                }
                f_k += cuts.of[f_p].kc();
                if (f_k >= f_depth) aim();
            }
            copy_commit();
        };
        aim();
#pragma unroll
        for (int i = 0; i < STAGES; ++i) fetch(i);

        int ws = 0, reds = 0;
        uint32_t rp = 0;
        bool on = true;
        int b_stage[2] = {0, 0};
        uint32_t b_phase[2] = {0, 0};
        typename L::Unit u;
        for (int at_unit = 0; on && unit_at(at_unit, u); ++at_unit) {
            const int p = u.p;
            const Cut cut = cuts.of[p];
            const int K = p == 0 ? a.H : a.F, KC = cut.kc();
            const int rg = warp >> cut.log_kg, kg = warp & (cut.kg() - 1), UP = cut.u() + 4;
            const int pitch = cut.b_pitch(), slot = cuts.b_rows * (p + 1) * pitch;
            const uint32_t b_first = b_ring + (p == 0 ? 0 : cuts.b_second) + kg * STAGE_COLS * 2, b_rest = cuts.b_rows * pitch;
            // A column past the last token takes any row that is there: nobody reads its sums.
            int b_row[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) b_row[t] = min(t * 8 + g, cuts.b_rows - 1) * pitch;
            int bs = b_stage[p];
            uint32_t bp = b_phase[p];
            const typename L::Entry en = entry[u.entry];
            const int tiles = (en.count + 7) >> 3;
            float acc[NT][CHAINS][4];   // sums of products that do not wait for one another
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4 * CHAINS; ++i) acc[t][i >> 2][i & 3] = 0.0f;
            uint32_t shift[2] = {0, 0};   // where a row's first value lies in its granule
            if (ODD) {
                const Rows r = rows_at(p, u.block, rg);
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    shift[i] = static_cast<uint32_t>((reinterpret_cast<uintptr_t>(p == 0 ? a.w1 : a.w2) +
                                                      (static_cast<int64_t>(en.expert) * rows_of[p] + r.first + g + i * (8 + r.jump)) * K * 2) & 15u);
            }
            for (int k0 = 0; k0 < K; k0 += KC) {
                copy_wait<STAGES - 1>();
                __syncwarp();
                const int n = min(KC, K - k0) - kg * STAGE_COLS;   // columns of this warp
                const uint32_t w_at = smem_u32(ring + ws * L::W_STAGE) + g * L::W_PITCH;
                uint4 a0[4], a1[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int col = q * 32 + c * 8;
                    a0[q] = a1[q] = make_uint4(0, 0, 0, 0);
                    if (col >= n) continue;
                    if (!ODD) {
                        const uint32_t from = w_at + ((q * 4 + c) ^ (g & 1) << 2) * 16;
                        a0[q] = lds128(from);
                        a1[q] = lds128(from + 8 * L::W_PITCH);
                    } else {
                        uint32_t v[2][4];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t from = w_at + 8 * i * L::W_PITCH + ((shift[i] + col * 2) & ~3u);
                            const uint32_t by = (shift[i] & 2u) * 8u;
                            uint32_t word[5];
#pragma unroll
                            for (int j = 0; j < 4; ++j) word[j] = lds32(from + 4 * j);
                            word[4] = by != 0 ? lds32(from + 16) : 0u;
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                // past the row's end is another row, or what the ring held before
                                const int left = n - col - 2 * j;
                                const uint32_t mask = left >= 2 ? 0xffffffffu : left == 1 ? 0xffffu : 0u;
                                v[i][j] = __funnelshift_r(word[j], word[j + 1], by) & mask;
                            }
                        }
                        a0[q] = make_uint4(v[0][0], v[0][1], v[0][2], v[0][3]);
                        a1[q] = make_uint4(v[1][0], v[1][1], v[1][2], v[1][3]);
                    }
                }
                __syncwarp();
                fetch(ws);   // the weights are in registers: their slot takes the next ones
                if (on) on = warp_wait(smem_u32(&s.b_full[p][bs]), bp, gave_up);
                if (on) {
                    const uint32_t b_at = b_first + bs * slot;
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        if (t >= tiles) break;
#pragma unroll
                        for (int half = 0; half < 2; ++half) {   // of h: the nearest values, and the rest
                            if (half > p) break;
                            uint4 b[4];
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const int col = q * 32 + c * 8;
                                b[q] = make_uint4(0, 0, 0, 0);
                                if (col < n) b[q] = lds128(b_at + (half ? b_rest : 0u) + b_row[t] + col * 2);
                            }
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                mma16816(acc[t][2 * q % CHAINS], a0[q].x, a1[q].x, a0[q].y, a1[q].y, b[q].x, b[q].y);
                                mma16816(acc[t][(2 * q + 1) % CHAINS], a0[q].z, a1[q].z, a0[q].w, a1[q].w, b[q].z, b[q].w);
                            }
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&s.b_empty[p][bs]));
                }
                if (++ws == STAGES) ws = 0;
                if (++bs == cut.b_stages) {
                    bs = 0;
                    bp ^= 1u;
                }
            }
            if (on) on = warp_wait(smem_u32(&s.red_empty[reds]), rp ^ 1u, gave_up);
            if (on) {
                float *const to = red + reds * L::RED;
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    if (t >= tiles) break;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        to[(kg * TOKENS + t * 8 + 2 * c + (i & 1)) * UP + rg * 16 + g + (i & 2 ? 8 : 0)] =
                            CHAINS == 4 ? (acc[t][0][i] + acc[t][1][i]) + (acc[t][2 % CHAINS][i] + acc[t][3 % CHAINS][i])
                                        : acc[t][0][i] + acc[t][1][i];
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&s.red_full[reds]));
            }
            if (++reds == cuts.reds) {
                reds = 0;
                rp ^= 1u;
            }
            b_stage[p] = bs;
            b_phase[p] = bp;
            unit_done(at_unit);
        }
        copy_wait<0>();
    } else {
        const int tid = threadIdx.x - MATH_THREADS - 64;
        int reds = 0;
        uint32_t rp = 0;
        for (int i = 0;; ++i) {
            typename L::Unit u;
            u.p = 0;
            bool on = unit_at(i, u);
            if (on) on = warp_wait(smem_u32(&s.red_full[reds]), rp, gave_up);
            if (!join_all(on)) break;   // both warps, or none: barriers follow
            const int p = u.p, block = u.block, KG = cuts.of[p].kg(), U = cuts.of[p].u(), UP = U + 4;
            const int log_u = 7 - cuts.of[p].log_kg, log_fu = log_u - (gated ? 1 : 0);
            const typename L::Entry en = entry[u.entry];
            const float *const from = red + reds * L::RED;
            // The warps' shares of the columns, in order.
            const auto joined = [&](int token, int row) {
                float v = from[token * UP + row];
#pragma unroll 2
                for (int k = 1; k < KG; ++k) v += from[(k * TOKENS + token) * UP + row];
                return v;
            };
            if (p == 0) {
                const mp_bf16_t *b1 = a.b1 == nullptr ? nullptr
                                                      : a.b1 + static_cast<int64_t>(en.expert) * a.F * (gated ? 2 : 1);
                for (int i = tid; i < FU * en.count; i += JOIN_THREADS) {
                    const int token = i >> log_fu, j = i & (FU - 1), f = block * FU + j;
                    if (f >= a.Fp) continue;
                    float h = 0.0f;   // up to a row's last 16 bytes
                    if (f < a.F) {
                        // Rows of the products: tiles of 8 of the gate and 8 of the other half.
                        h = joined(token, gated ? (j >> 3) * 16 + (j & 7) : j);
                        if (b1 != nullptr) h += bf16_value(b1 + f);
                        h = act_of(a.act, h);
                        if (gated) {
                            float o = joined(token, (j >> 3) * 16 + (j & 7) + 8);
                            if (b1 != nullptr) o += bf16_value(b1 + a.F + f);
                            h *= o;
                        }
                    }
                    mp_bf16_t *const to = a.h + static_cast<int64_t>(order[en.first + token]) * 2 * a.Fp + f;
                    const float value[1] = {h};
                    const mp_bf16_t near = pack(value);
                    float back[1];
                    unpack(near, back);
                    const float rest[1] = {isfinite(back[0]) ? h - back[0] : 0.0f};
                    to[0] = near;
                    to[a.Fp] = pack(rest);
                }
            } else {
                const mp_bf16_t *b2 = a.b2 == nullptr ? nullptr : a.b2 + static_cast<int64_t>(en.expert) * a.O;
                for (int i = tid; i < U * en.count; i += JOIN_THREADS) {
                    const int token = i >> log_u, j = i & (U - 1), o = block * U + j;
                    if (o >= a.O) continue;
                    float v = joined(token, j);
                    if (b2 != nullptr) v += bf16_value(b2 + o);
                    a.out[static_cast<int64_t>(order[en.first + token]) * a.O + o] = v;
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&s.red_empty[reds]));
            if (p == 0) {   // h of this unit is there for the copies of all SMs
                fence_async();
                __threadfence();
                join_barrier();
                if (tid == 0) grid_arrive(&a.control->done[u.entry]);
            }
            if (++reds == cuts.reds) {
                reds = 0;
                rp ^= 1u;
            }
            unit_done(i);
        }
        // What this CTA made is there for the others.
        __threadfence();
        join_barrier();
        if (tid == 0) grid_arrive(&a.control->arrived[1]);
        if (tid == 0) (void)grid_wait(&a.control->arrived[1], gridDim.x, gave_up);
    }
    most_barrier();
    constexpr int LEFT = MATH_THREADS + JOIN_THREADS;
    const int tid = threadIdx.x < MATH_THREADS ? threadIdx.x : threadIdx.x - 64;
    // The slots of each token, in order; four columns a thread where rows of sums are whole 16 bytes.
    const int wide = a.O % 4 == 0 ? 4 : 1, across = a.O / wide;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * LEFT + tid; i < static_cast<int64_t>(a.T) * across;
         i += static_cast<int64_t>(gridDim.x) * LEFT) {
        const int t = static_cast<int>(i / across), o = static_cast<int>(i - static_cast<int64_t>(t) * across) * wide;
        const float *const from = a.out + static_cast<int64_t>(t) * a.K * a.O + o;
        float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int k0 = 0; k0 < a.K; k0 += 8) {   // eight loads at a time
            float4 v[8];
            float w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const bool there = k0 + k < a.K && idx[t * a.K + k0 + k] >= 0;
                const float *const at = from + static_cast<int64_t>(k0 + k) * a.O;
                w[k] = there ? weights[t * a.K + k0 + k] : 0.0f;
                v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (there && wide == 4) v[k] = __ldcg(reinterpret_cast<const float4 *>(at));
                if (there && wide == 1) v[k].x = __ldcg(at);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {   // a slot that is not there adds 0 times 0
                y[0] = fmaf(w[k], v[k].x, y[0]);
                y[1] = fmaf(w[k], v[k].y, y[1]);
                y[2] = fmaf(w[k], v[k].z, y[2]);
                y[3] = fmaf(w[k], v[k].w, y[3]);
            }
        }
        mp_bf16_t *const to = a.y + static_cast<int64_t>(t) * a.O + o;
        for (int j = 0; j < wide; ++j) {
            const float v[1] = {y[j]};
            to[j] = pack(v);
        }
    }
    if (tid == 0 && *gave_up) or_status(a.status, MP_STATUS_STALLED);
}

template <typename L> void launch_logits(const LayerArgs &a, cudaStream_t s)
{
    const bool vec = a.H % 4 == 0 && reinterpret_cast<uintptr_t>(a.x) % 8 == 0 &&
                     reinterpret_cast<uintptr_t>(a.router) % (4 * sizeof(L)) == 0;
    const unsigned E = static_cast<unsigned>(a.E);
    if (a.T <= 2)
        (void)launch_pdl(vec ? k_layer_logits<L, 1, true> : k_layer_logits<L, 1, false>, dim3(E, a.T), LOGIT_THREADS, 0, s, a);
    else
        (void)launch_pdl(vec ? k_layer_logits<L, 4, true> : k_layer_logits<L, 4, false>, dim3(E, (a.T + 3) / 4),
                         LOGIT_THREADS, 0, s, a);
}

// The cut of a product of `rows` by `depth`, of `entries` entries: the fewest cycles by this count.
// A stage of 32 KB takes 1,400 cycles at the copy bandwidth and more with many tokens' rows beside
// it (which it reads for U rows each), a unit's end 800.  (Rows that start anywhere take more of the
// first; they are counted alike.)  Columns that a stage has and the product
// has not are idle warps.  At the end SMs wait for the last units, and at the start of the second
// product for about half a unit of the first (`late`).  One token through 8 experts of 1,024 x
// 4,096, U of the first and second product: 128, 128 57.8 us; 64, 64 51.3; 32, 64 47.5; 32, 32 47.9;
// 16, 32 50.4.  8 tokens through 57 of 512 x 7,168: 32, 128 209; 32, 64 221; 32, 32 246.
Cut cut_product(int64_t entries, int rows, int depth, double tokens, int most_log, double late)
{
    Cut best = {0, 0};
    double least = 0;
    for (int log = 0; log <= most_log; ++log) {
        const Cut c = {log, 0};
        const int64_t units = entries * ((rows + c.u() - 1) / c.u()), stages = (depth + c.kc() - 1) / c.kc();
        const double unit = static_cast<double>(stages) * 1400.0 * (1.0 + tokens / c.u()) + 800.0;
        const double cycles = unit * (static_cast<double>(units) / sm_count() + late);
        if (log == 0 || cycles < least) {
            best = c;
            least = cycles;
        }
    }
    return best;
}

template <int NT, bool ODD> mp_status_t launch_layer(const LayerArgs &a, cudaStream_t s)
{
    typedef Layer<NT, ODD> L;
    static std::atomic<uint64_t> allowed{0};
    if (!allow_smem(k_layer<NT, ODD>, allowed, LAYER_SMEM)) return MP_ERR_CUDA;
    const int R = a.T * a.K;
    const bool gated = act_gated(a.act);
    // Experts that are picked, if all are alike: E (1 - (1 - K / E)^T).
    double missed = 1.0;
    for (int t = 0; t < a.T; ++t) missed *= 1.0 - static_cast<double>(a.K) / a.E;
    const double busy = a.E * (1.0 - missed), tokens = R / busy;
    const int64_t entries = static_cast<int64_t>(busy * ((tokens + L::TOKENS - 1) / L::TOKENS > 1.5 ? 2 : 1) + 0.5);
    // So that slots for the tokens' rows fit: two or more of each product but with the largest tables.
    constexpr int most_log[2] = {NT == 1 ? 3 : NT == 2 ? 1 : 0, NT == 1 ? 2 : NT == 2 ? 1 : 0};
    LayerCuts cuts;
    cuts.of[0] = cut_product(entries, a.F * (gated ? 2 : 1), a.H, tokens, most_log[0], 0.5);
    cuts.of[1] = cut_product(entries, a.O, a.F, 2.0 * tokens, most_log[1], 1.0);
    cuts.b_rows = a.T < L::TOKENS ? a.T : L::TOKENS;
    const size_t fixed = L::tables(a.E, R) + static_cast<size_t>(L::STAGES) * L::W_STAGE;
    const size_t slots[2] = {static_cast<size_t>(cuts.b_rows) * cuts.of[0].b_pitch(),
                             static_cast<size_t>(cuts.b_rows) * 2 * cuts.of[1].b_pitch()};
    for (cuts.reds = RED_MOST; cuts.reds > 1 && fixed + cuts.reds * L::RED * 4 + 2 * (slots[0] + slots[1]) > LAYER_SMEM; --cuts.reds) {
    }
    // (1,024 experts and 2,048 routes leave room for one slot of each.)
    size_t bytes = fixed + static_cast<size_t>(cuts.reds) * L::RED * 4 + slots[0] + slots[1];
    int n[2] = {1, 1};
    for (bool more = true; more;) {   // of the product with fewer, as long as there is room
        more = false;
        for (int i = 0; i < 2 && !more; ++i) {
            const int p = (n[1] < n[0]) ^ (i == 1);
            if (n[p] < B_MOST && bytes + slots[p] <= LAYER_SMEM) {
                bytes += slots[p];
                ++n[p];
                more = true;
            }
        }
    }
    cuts.of[0].b_stages = n[0];
    cuts.of[1].b_stages = n[1];
    cuts.b_second = static_cast<int>(n[0] * slots[0]);
    const int room = static_cast<int>(n[0] * slots[0] + n[1] * slots[1]);
    // No more CTAs than units: a barrier of few is quicker.
    const int64_t most = (a.E < R ? a.E : R) + R / L::TOKENS;
    int64_t wide = 0;
    for (int p = 0; p < 2; ++p) {
        const int rows = p == 0 ? a.F * (gated ? 2 : 1) : a.O, u = cuts.of[p].u();
        if ((rows + u - 1) / u > wide) wide = (rows + u - 1) / u;
    }
    const int sms = sm_count();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = static_cast<unsigned>(most * wide < sms ? most * wide : sms);
    cfg.blockDim = LAYER_THREADS;
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    (void)cudaLaunchKernelEx(&cfg, k_layer<NT, ODD>, a, cuts, room);
    return check_launch();
}

// Up to 8, 16 or 32 tokens an entry.  An expert with more than 16 has its weights copied once with 32 an entry and
// twice with 16; but such a unit is 128 rows, which share the SMs badly where experts are few.  64 tokens, 64 experts of
// 1,024 x 2,048, 12, 14, 16, 24, 32 tokens an expert, us with 16 and 32: 190, 199; 220, 212; 251, 224; 341, 277; 422, 387.
// 32 experts, 12, 16: 111, 117; 142, 129.  16 experts of 512 x 4,096, 14, 20, 26: 84, 100; 117, 117; 122, 136; 8
// experts, 12, 32: 62, 76; 89, 122.
template <bool ODD> mp_status_t choose_layer(const LayerArgs &a, cudaStream_t s)
{
    if (a.T <= 8) return launch_layer<1, ODD>(a, s);
    if (a.E < 32 || a.T * a.K <= 12 * a.E) return launch_layer<2, ODD>(a, s);
    return launch_layer<4, ODD>(a, s);
}

mp_status_t layer_sizes(int64_t T, int32_t E, int32_t K, int32_t H, int32_t F, int32_t O)
{
    if (T < 0 || E < 1 || K < 1 || K > E || H < 1 || F < 1 || O < 1) return MP_ERR_INVALID_ARG;
    constexpr int WIDEST = MP_MAX_LAYER_WIDTH;
    return T > MP_MAX_LAYER_TOKENS || E > MP_MAX_EXPERTS || K > 32 || H > WIDEST || F > WIDEST || O > WIDEST
               ? MP_ERR_UNSUPPORTED
               : MP_OK;
}

int whole(int n) { return (n + 7) / 8 * 8; }

// Where the parts of the workspace start, in bytes; the last is its size.
struct LayerSpace {
    size_t logits, xp, h, out, bytes;
    LayerSpace(int64_t T, int64_t E, int64_t K, int H, int F, int64_t O)
    {
        const auto next = [](size_t from, size_t bytes) { return (from + bytes + 255) / 256 * 256; };
        logits = next(0, sizeof(LayerControl));
        xp = next(logits, static_cast<size_t>(T * E) * 4);
        h = next(xp, static_cast<size_t>(T) * whole(H) * 2);
        out = next(h, static_cast<size_t>(T * K) * whole(F) * 4);
        bytes = next(out, static_cast<size_t>(T * K * O) * 4);
    }
};

}  // namespace
}  // namespace mp

using namespace mp;

extern "C" size_t mp_moe_layer_workspace_size(int64_t T, int32_t E, int32_t K, int32_t H, int32_t F, int32_t O)
{
    return layer_sizes(T, E, K, H, F, O) != MP_OK ? 0 : LayerSpace(T, E, K, H, F, O).bytes;
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
    const LayerSpace space(T, E, K, H, F, O);
    if (workspace == nullptr || !aligned16(workspace) || workspace_bytes < space.bytes) return MP_ERR_WORKSPACE;
    uint8_t *const ws = static_cast<uint8_t *>(workspace);
    const cudaStream_t s = as_stream(stream);
    route.T = T; route.idx = idx; route.weights = weights;
    LayerArgs a = {};
    a.x = x; a.w1 = w1; a.b1 = b1; a.w2 = w2; a.b2 = b2; a.router = router; a.route = route;
    a.T = static_cast<int>(T); a.E = E; a.K = K; a.H = H; a.F = F; a.O = O; a.act = act;
    a.idx = idx; a.weights = weights; a.y = y; a.status = dev_status;
    a.control = reinterpret_cast<LayerControl *>(ws);
    a.logits = reinterpret_cast<float *>(ws + space.logits);
    a.Hp = whole(H); a.Fp = whole(F);
    a.xp = H % 8 == 0 && aligned16(x) ? nullptr : reinterpret_cast<mp_bf16_t *>(ws + space.xp);
    a.h = reinterpret_cast<mp_bf16_t *>(ws + space.h);
    a.out = reinterpret_cast<float *>(ws + space.out);
    switch (router_dtype) {
    case MP_DTYPE_BF16: launch_logits<__nv_bfloat16>(a, s); break;
    case MP_DTYPE_FP16: launch_logits<__half>(a, s); break;
    default: launch_logits<float>(a, s); break;
    }
    if (const mp_status_t st = check_launch(); st != MP_OK) return st;
    const bool even = H % 8 == 0 && F % 8 == 0 && aligned16(w1) && aligned16(w2);
    return even ? choose_layer<false>(a, s) : choose_layer<true>(a, s);
}
