// The router of current mixture models: softmax or sigmoid scores, a bias for
// balance, groups of experts, top-K, renormalised weights; and its gradient.
//
//   s_e = softmax(l)_e or sigmoid(l_e);  c_e = s_e + b_e decides the choice
//   weights: scale * s_k / sum_j s_j (renorm) or scale * s_k
//
// k_route: one warp per token; lane l holds the experts l, l+32, ...
// Choice.  Without a bias the scores rise with the logits, which are compared
// as they are.  With one, and for the sum of a group's best two, fp32 values of
// c decide wherever neighbours in the order are further apart than their errors
// can be (too_near); a token where two are nearer (about one of two thousand of
// normal logits) is decided again in 64 bits: the two groups or the picks and the best
// of the rest where that is enough, else everything (choose_exact).  So the choice is
// that of 64 bits everywhere, at the cost of 32: on 32,768 tokens of 256 experts
// (sigmoid, bias, 8 groups), all of it in 64 bits took 1,290 us, this 39 (43 with choose_exact for all near tokens).
// Each lane sorts its candidates by a fixed network and a round takes the best
// head of the warp (topk.cuh); the round after the K-th says how near the best
// of the rest is.
// Weights are fp32 from the picks' own logits.
// k_route_bwd: one warp per token; every gradient is written once.
#include <cfloat>
#include <cuda_fp16.h>

#include "topk.cuh"

namespace mp {
namespace {

constexpr int RT_THREADS = 256;
constexpr int RT_WARPS = RT_THREADS / 32;

struct RouteArgs {
    const void *logits;
    const float *bias;
    int64_t T;
    int E, K, score, n_groups, topk_groups, group_top, renorm;
    uint32_t group_magic;   // ceil(2^32 / experts a group): (e * magic) >> 32 is e's group (of 2 experts or more)
    float scale;
    int32_t *idx;
    float *weights;
};

__device__ __forceinline__ float logit(const float *p) { return __ldg(p); }
__device__ __forceinline__ float logit(const __nv_bfloat16 *p)
{
    return __uint_as_float(static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t *>(p))) << 16);
}
__device__ __forceinline__ float logit(const __half *p) { return __half2float(__ldg(p)); }
__device__ __forceinline__ float logit_value(float v) { return v; }
__device__ __forceinline__ float logit_value(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float logit_value(__half v) { return __half2float(v); }

__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(__half *p, float v) { *p = __float2half_rn(v); }

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL_MASK, v, d));
    return v;
}
template <typename F> __device__ __forceinline__ F warp_sum(F v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(FULL_MASK, v, d);
    return v;
}

using mp::key_value;
using mp::order_key;
using mp::warp_argmax_key;

// order_key in 64 bits: 0 stands for no candidate.
__device__ __forceinline__ uint64_t order_key(double d)
{
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(d + 0.0));   // -0 becomes +0
    return u ^ (static_cast<uint64_t>(static_cast<int64_t>(u) >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double key_value(uint64_t k)
{
    return __longlong_as_double(
        static_cast<int64_t>((k >> 63) ? k & 0x7fffffffffffffffull : ~k));
}
// Arg-max on (key desc, index asc); every lane gets both.
__device__ __forceinline__ uint32_t warp_argmax_key(uint64_t &key, uint32_t idx)
{
    const uint32_t hi = static_cast<uint32_t>(key >> 32), lo = static_cast<uint32_t>(key);
    const uint32_t mh = __reduce_max_sync(FULL_MASK, hi);
    const uint32_t ml = __reduce_max_sync(FULL_MASK, hi == mh ? lo : 0u);
    const uint32_t i = __reduce_min_sync(FULL_MASK, hi == mh && lo == ml ? idx : 0xffffffffu);
    key = static_cast<uint64_t>(mh) << 32 | ml;
    return i;
}

// The same over lanes 0..K-1 of a token of KT picks (0: any): with KT a power of
// two below 32, lanes 0..KT-1 reduce among themselves.
template <int KT> __device__ __forceinline__ float pick_max(float v)
{
#pragma unroll
    for (int d = KT > 0 ? KT / 2 : 16; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL_MASK, v, d));
    return v;
}
template <int KT> __device__ __forceinline__ float pick_sum(float v)
{
#pragma unroll
    for (int d = KT > 0 ? KT / 2 : 16; d; d >>= 1) v += __shfl_xor_sync(FULL_MASK, v, d);
    return v;
}

// A logit that can be chosen: not -inf and not NaN (an unavailable expert);
// +inf counts as the largest finite value.
__device__ __forceinline__ bool usable(float v) { return v > -INFINITY; }


// The token's logits and biases: expert lane + 32 j in slot j.  What cannot be
// chosen has logit -inf; +inf is the largest finite value.
template <typename L, int PER>
__device__ __forceinline__ void load_token(const RouteArgs &a, const L *l, int lane, float (&v)[PER],
                                           float (&b)[PER])
{
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int e = lane + 32 * j;
        v[j] = e < a.E ? logit(l + e) : -INFINITY;
        b[j] = (e < a.E && a.bias != nullptr) ? __ldg(a.bias + e) : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) v[j] = usable(v[j]) ? fminf(v[j], FLT_MAX) : -INFINITY;   // NaN is not usable
}

// exp(-x) for x >= 0 in 64 bits, within 2 units of the last place: x = n ln 2 + r
// by a reduction in two steps (Cody and Waite), Taylor's series of exp(-r), |r| <= ln 2 / 2,
// to r^13 (the next term is 4e-18).  Without branches, so that a lane's values
// are worked on side by side: the units for 64 bits are few, and what counts is the
// length of the chain (one token of 256 experts: 18 us with exp(), 6 with this).
__device__ __forceinline__ double exp_neg(double x)
{
    x = fmin(x, 745.0);
    const double n = rint(x * 1.4426950408889634074);
    double r = fma(n, -0.6931471796706319, x);   // ln 2 cut off after 30 bits: the product is exact
    r = -fma(n, -8.893134238886677e-10, r);           // and what was cut off
    double s = 1.0 / 6227020800.0;
    s = fma(s, r, 1.0 / 479001600.0);
    s = fma(s, r, 1.0 / 39916800.0);
    s = fma(s, r, 1.0 / 3628800.0);
    s = fma(s, r, 1.0 / 362880.0);
    s = fma(s, r, 1.0 / 40320.0);
    s = fma(s, r, 1.0 / 5040.0);
    s = fma(s, r, 1.0 / 720.0);
    s = fma(s, r, 1.0 / 120.0);
    s = fma(s, r, 1.0 / 24.0);
    s = fma(s, r, 1.0 / 6.0);
    s = fma(s, r, 0.5);
    s = fma(s, r, 1.0);
    s = fma(s, r, 1.0);
    // 2^-n in two factors, so that the smallest results come out rounded once.
    const int k = static_cast<int>(n), h = k >> 1;
    const double p = __longlong_as_double(static_cast<long long>(1023 - h) << 52);
    const double q = __longlong_as_double(static_cast<long long>(1023 - (k - h)) << 52);
    return s * p * q;
}

// 1/x for 1 <= x <= 2^11: an fp32 reciprocal and two steps of Newton's, each of which
// squares the error.
__device__ __forceinline__ double rcp_exact(double x)
{
    double r = static_cast<double>(__frcp_rn(static_cast<float>(x)));
    r = fma(r, fma(-x, r, 1.0), r);
    return fma(r, fma(-x, r, 1.0), r);
}

// A score that decides, in 64 bits: for softmax without the common divisor, and so
// only where there is no bias.  `m`: the largest logit (softmax).  0: cannot be chosen.
template <typename L>
__device__ __forceinline__ uint64_t exact_key(const RouteArgs &a, const L *l, int e, float m)
{
    const float v = logit(l + e), b = a.bias != nullptr ? __ldg(a.bias + e) : 0.0f;
    if (!usable(v) || !usable(b)) return 0ull;
    const double x = fminf(v, FLT_MAX);
    double c;
    if (a.score == MP_SCORE_SIGMOID) {
        const double t = exp_neg(fabs(x));
        c = (x < 0.0 ? t : 1.0) * rcp_exact(1.0 + t);
    } else {
        c = exp_neg(static_cast<double>(m) - x);
    }
    return order_key(c + static_cast<double>(b));
}

// Whether group gb stands before ga in 64 bits, by the sum of their best one or two.
template <typename L>
__device__ __noinline__ bool groups_turned(const RouteArgs &a, const L *l, int lane, int ga, int gb)
{
    float m = -INFINITY;
    if (a.score == MP_SCORE_SOFTMAX) {
        for (int e = lane; e < a.E; e += 32) m = fmaxf(m, fminf(logit(l + e), FLT_MAX));   // NaN is passed over
        m = warp_max(m);
    }
    const int n = a.E / a.n_groups;
    uint64_t worth[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        uint64_t k1 = 0ull, k2 = 0ull;
        for (int i = lane; i < n; i += 32) {
            const uint64_t k = exact_key(a, l, (q ? gb : ga) * n + i, m);
            k2 = max(k2, min(k, k1));
            k1 = max(k1, k);
        }
        uint64_t w = k1;
        const uint32_t holder = warp_argmax_key(w, static_cast<uint32_t>(lane));
        if (a.group_top == 2) {
            uint64_t m2 = lane == holder ? k2 : k1;
            (void)warp_argmax_key(m2, static_cast<uint32_t>(lane));
            if (m2 != 0ull) w = order_key(key_value(w) + key_value(m2));
        }
        worth[q] = w;
    }
    return worth[1] > worth[0] || (worth[1] == worth[0] && gb < ga);
}

// Orders the experts of lanes 0..K (-1: none) in 64 bits; lane k < K gets the k-th.
template <typename L>
__device__ __noinline__ int picks_in_order(const RouteArgs &a, const L *l, int lane, int K, int expert)
{
    const uint64_t key = expert >= 0 ? exact_key(a, l, expert, 0.0f) : 0ull;
    int rank = 0, got = -1;
    for (int j = 0; j <= K; ++j) {
        const uint64_t k = __shfl_sync(FULL_MASK, key, j);
        const int e = __shfl_sync(FULL_MASK, expert, j);
        rank += k > key || (k == key && e < expert);
    }
    for (int j = 0; j <= K; ++j) {
        const int at = __shfl_sync(FULL_MASK, rank, j), e = __shfl_sync(FULL_MASK, expert, j);
        if (at == lane && e >= 0) got = e;
    }
    return lane < K ? got : -1;
}

// The choice in 64 bits.  Lane k gets pick k (-1: none left).
template <typename L, int PER>
__device__ __noinline__ int choose_exact(const RouteArgs &a, const L *l, int lane)
{
    float v[PER], b[PER];
    load_token<L, PER>(a, l, lane, v, b);
    double c[PER];
    if (a.score == MP_SCORE_SIGMOID) {
        // 1 / (1 + exp(-v)), with the exponential of -|v|.
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const double t = exp_neg(fabs(static_cast<double>(v[j])));
            c[j] = (v[j] < 0.0f ? t : 1.0) * rcp_exact(1.0 + t);
        }
    } else {
        float m = -INFINITY;
#pragma unroll
        for (int j = 0; j < PER; ++j) m = fmaxf(m, v[j]);
        m = warp_max(m);
        double s = 0.0;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            c[j] = usable(v[j]) ? exp_neg(static_cast<double>(m) - v[j]) : 0.0;
            s += c[j];
        }
        s = rcp_exact(fmax(warp_sum(s), 1.0));   // the largest term is 1, if there is any
#pragma unroll
        for (int j = 0; j < PER; ++j) c[j] *= s;
    }
    uint64_t key[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j)
        key[j] = usable(v[j]) && usable(b[j]) ? order_key(c[j] + static_cast<double>(b[j])) : 0ull;
    if (a.n_groups > 1) {
        uint64_t worth = 0ull;   // lane g: group g's
        for (int g = 0; g < a.n_groups; ++g) {
            uint64_t k1 = 0ull, k2 = 0ull;
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const uint64_t k = __umulhi(lane + 32 * j, a.group_magic) == g ? key[j] : 0ull;
                k2 = max(k2, min(k, k1));
                k1 = max(k1, k);
            }
            uint64_t w = k1;
            const uint32_t holder = warp_argmax_key(w, static_cast<uint32_t>(lane));
            if (a.group_top == 2) {
                uint64_t m2 = lane == holder ? k2 : k1;
                (void)warp_argmax_key(m2, static_cast<uint32_t>(lane));
                if (m2 != 0ull) w = order_key(key_value(w) + key_value(m2));
            }
            if (lane == g) worth = w;
        }
        unsigned kept = 0;
        for (int r = 0; r < a.topk_groups; ++r) {
            uint64_t wk = (kept >> lane & 1u) ? 0ull : worth;
            const uint32_t g = warp_argmax_key(wk, static_cast<uint32_t>(lane));
            if (wk != 0ull) kept |= 1u << g;
        }
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if (!(kept >> (__umulhi(lane + 32 * j, a.group_magic) & 31) & 1u)) key[j] = 0ull;
    }
    // Without a bias the scores rise with the logits, which stay apart where
    // scores round to one value.
#pragma unroll
    for (int j = 0; j < PER; ++j)
        if (a.bias == nullptr && key[j] != 0ull) key[j] = order_key(static_cast<double>(v[j]));
    int pick = -1;
    for (int k = 0; k < a.K; ++k) {
        uint64_t bk = 0ull;
        uint32_t bi = 0xffffffffu;
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if (key[j] > bk) {
                bk = key[j];
                bi = static_cast<uint32_t>(lane + 32 * j);
            }
        const uint32_t p = warp_argmax_key(bk, bi);
        if (bk == 0ull) break;
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if (lane + 32 * j == p) key[j] = 0ull;
        if (lane == k) pick = static_cast<int>(p);
    }
    return pick;
}

// 2^(x log2 e) and 1/x of the special function unit: within 2 ulp, plus the
// rounding of the argument.
__device__ __forceinline__ float exp_fast(float x) { return __expf(x); }
__device__ __forceinline__ float rcp_fast(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ void into_top2(uint32_t k, uint32_t &k1, uint32_t &k2)
{
    k2 = max(k2, min(k, k1));
    k1 = max(k1, k);
}

// Picks by 32-bit keys, 0 for none.  Lane k gets pick k's key and expert; `rest`
// and `rest_i` are those of the best of the rest, `after` the key of the next.
template <int N, int KT>
__device__ __forceinline__ void rounds(uint32_t (&key)[N], uint32_t (&ex)[N], int K, int lane,
                                       uint32_t &my_key, int &my_i, uint32_t &rest, uint32_t &rest_i,
                                       uint32_t &after)
{
    sort_desc<N>(key, ex);
    if (KT > 0) K = KT;
#pragma unroll
    for (int k = 0; k < (KT > 0 ? KT : K); ++k) {
        uint32_t bk = key[0];
        const uint32_t pick = warp_argmax_key(bk, ex[0]);
        if (ex[0] == pick) {
#pragma unroll
            for (int j = 0; j + 1 < N; ++j) {
                key[j] = key[j + 1];
                ex[j] = ex[j + 1];
            }
            key[N - 1] = 0u;
        }
        if (lane == k) {
            my_key = bk;
            my_i = static_cast<int>(pick);
        }
    }
    rest = key[0];
    rest_i = warp_argmax_key(rest, ex[0]);
    after = __reduce_max_sync(FULL_MASK, ex[0] == rest_i ? key[1] : key[0]);
}

// Whether two values next to each other in a descending order, each off by at
// most err + 2^-24 of its magnitude, may belong the other way round.
__device__ __forceinline__ bool too_near(uint32_t key, uint32_t next, float err)
{
    if (key == 0u || next == 0u) return false;
    const float c = key_value(key), d = key_value(next);
    return !(c - d > 2.0f * err + 6.0e-8f * (fabsf(c) + fabsf(d)));
}

// The choice from fp32 values; false (in every lane): too near to tell.
template <typename L, int PER, int KT>
__device__ __forceinline__ bool choose_fast(const RouteArgs &a, const L *l, const float (&v)[PER],
                                            const float (&b)[PER], int lane, int &pick)
{
    const int K = KT > 0 ? KT : a.K;
    const bool by_logit = a.bias == nullptr;
    const bool pairs = a.n_groups > 1 && a.group_top == 2;
    uint32_t key[PER];
    float err = 0.0f;   // absolute error of a score
    bool near = false;
    if (!by_logit || pairs) {
        // sigmoid: exp within (2 + |v|) ulp, its share of the result s (1 - s),
        // then a sum and a reciprocal: 3e-7 of 1.  softmax: the largest score
        // times the same, the argument's rounding and the sum of E terms.
        float c[PER];
        if (a.score == MP_SCORE_SIGMOID) {
            err = 4e-7f;
#pragma unroll
            for (int j = 0; j < PER; ++j) c[j] = rcp_fast(1.0f + exp_fast(-v[j]));
        } else {
            float m = -INFINITY, sum = 0.0f;
#pragma unroll
            for (int j = 0; j < PER; ++j) m = fmaxf(m, v[j]);
            m = fmaxf(warp_max(m), -FLT_MAX);
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                c[j] = exp_fast(v[j] - m);   // 0 for -inf
                sum += c[j];
            }
            const float inv = rcp_fast(fmaxf(warp_sum(sum), 1.0f));
            err = inv * (8e-7f + (PER + 6) * 6e-8f);
#pragma unroll
            for (int j = 0; j < PER; ++j) c[j] *= inv;
        }
#pragma unroll
        for (int j = 0; j < PER; ++j)
            key[j] = usable(v[j]) && usable(b[j]) ? order_key(c[j] + b[j]) : 0u;
    } else {
#pragma unroll
        for (int j = 0; j < PER; ++j) key[j] = usable(v[j]) ? order_key(v[j]) : 0u;
    }

    unsigned cols = 0u;   // slots that may hold a candidate, the same in every lane
    if (a.n_groups > 1) {
        const int per_group = a.E / a.n_groups;
        const bool columns = per_group % 32 == 0;   // a group is whole slots
        uint32_t w1 = 0u, w2 = 0u;                  // lane g: group g's best two
        // From each lane's best two of group g.
        const auto finish = [&](int g, uint32_t k1, uint32_t k2) {
            const uint32_t m1 = __reduce_max_sync(FULL_MASK, k1);
            uint32_t m2 = 0u;
            if (a.group_top == 2) {
                m2 = __reduce_max_sync(FULL_MASK, k1 == m1 ? k2 : k1);
                if (__popc(__ballot_sync(FULL_MASK, k1 == m1)) > 1) m2 = m1;   // two lanes hold it
            }
            if (lane == g) {
                w1 = m1;
                w2 = m2;
            }
        };
        if (columns) {
            const int slots = per_group / 32;
            uint32_t k1 = 0u, k2 = 0u;
            int n = 0, g = 0;
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                into_top2(key[j], k1, k2);
                if (++n == slots && g < a.n_groups) {
                    finish(g, k1, k2);
                    k1 = k2 = 0u;
                    n = 0;
                    ++g;
                }
            }
        } else {
            for (int g = 0; g < a.n_groups; ++g) {
                uint32_t k1 = 0u, k2 = 0u;
#pragma unroll
                for (int j = 0; j < PER; ++j)
                    into_top2(__umulhi(lane + 32 * j, a.group_magic) == g ? key[j] : 0u, k1, k2);
                finish(g, k1, k2);
            }
        }
        const uint32_t worth = w2 == 0u ? w1 : order_key(key_value(w1) + key_value(w2));
        const float size = w2 == 0u ? 0.0f : fabsf(key_value(w1)) + fabsf(key_value(w2));
        // A group is kept if fewer than topk_groups stand before it.
        int before = 0;
        for (int g = 0; g < a.n_groups; ++g) {
            const uint32_t o = __shfl_sync(FULL_MASK, worth, g);
            before += o > worth || (o == worth && g < lane);
        }
        const bool mine = worth != 0u && before < a.topk_groups;
        unsigned kept = __ballot_sync(FULL_MASK, mine);
        if (err > 0.0f) {
            // Only the last one kept and the first one left out must stand apart.
            const uint32_t last = __reduce_min_sync(FULL_MASK, mine ? worth : 0xffffffffu);
            const uint32_t next = __reduce_max_sync(FULL_MASK, mine ? 0u : worth);
            const float slack = __uint_as_float(__reduce_max_sync(FULL_MASK, __float_as_uint(size)));
            const float off = 2.0f * err + 1.2e-7f * slack;
            near = kept != 0u && too_near(last, next, off);
            if (near && (by_logit || a.score == MP_SCORE_SIGMOID)) {
                // Mostly it is these two alone.
                const unsigned set = __ballot_sync(
                    FULL_MASK, worth != 0u && (mine ? too_near(worth, next, off) : too_near(last, worth, off)));
                if (__popc(set) == 2) {
                    if (groups_turned(a, l, lane, __ffs(set & kept) - 1, __ffs(set & ~kept) - 1)) kept ^= set;
                    near = false;
                }
            }
        }
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const unsigned in = kept >> (__umulhi(columns ? 32 * j : lane + 32 * j, a.group_magic) & 31) & 1u;
            key[j] = in ? key[j] : 0u;
            if (!columns || in) cols |= 1u << j;
        }
    } else {
        cols = (1u << (PER - 1) << 1) - 1u;
    }
    if ((a.E + 31) / 32 < PER) cols &= (1u << ((a.E + 31) / 32)) - 1u;
    if (by_logit && pairs) {   // without a bias the logits decide inside the groups
#pragma unroll
        for (int j = 0; j < PER; ++j) key[j] = key[j] ? order_key(v[j]) : 0u;
    }
    uint32_t ex[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) ex[j] = static_cast<uint32_t>(lane + 32 * j);
    uint32_t my_key = 0u, rest = 0u, rest_i = 0u, after = 0u;
    int my_i = -1;
    if constexpr (PER <= 8) {
        if (PER >= 4 && __popc(cols) <= PER / 2) {
            constexpr int HALF = PER >= 4 ? PER / 2 : 1;
            uint32_t kc[HALF], xc[HALF];
#pragma unroll
            for (int i = 0; i < HALF; ++i) {
                kc[i] = 0u;
                xc[i] = 0xffffffffu;
            }
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (cols >> j & 1u) {
#pragma unroll
                    for (int i = HALF - 1; i > 0; --i) {
                        kc[i] = kc[i - 1];
                        xc[i] = xc[i - 1];
                    }
                    kc[0] = key[j];
                    xc[0] = ex[j];
                }
            rounds<HALF, KT>(kc, xc, K, lane, my_key, my_i, rest, rest_i, after);
        } else {
            rounds<PER, KT>(key, ex, K, lane, my_key, my_i, rest, rest_i, after);
        }
    } else {
        // More than 256 experts: each round looks through the lane's own again.
        for (int k = 0; k <= K; ++k) {
            uint32_t bk = 0u, bi = 0xffffffffu;
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (key[j] > bk) {
                    bk = key[j];
                    bi = ex[j];
                }
            const uint32_t p = warp_argmax_key(bk, bi);
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (ex[j] == p) key[j] = 0u;
            if (lane == k && k < K) {
                my_key = bk;
                my_i = static_cast<int>(p);
            }
            rest = bk;
            rest_i = p;
        }
#pragma unroll
        for (int j = 0; j < PER; ++j) after = max(after, key[j]);
        after = __reduce_max_sync(FULL_MASK, after);
    }
    pick = (lane < K && my_key != 0u) ? my_i : -1;
    if (!by_logit) {
        // Neighbours of the same logit and bias are equal in any arithmetic,
        // and stand in the order of their indices already.
        uint32_t next = __shfl_down_sync(FULL_MASK, my_key, 1);
        uint32_t next_i = __shfl_down_sync(FULL_MASK, static_cast<uint32_t>(my_i), 1);
        if (lane == K - 1) {
            next = rest;
            next_i = rest_i;
        }
        bool unsure = false;
        if (lane < K && too_near(my_key, next, err))
            unsure = !(logit(l + my_i) == logit(l + next_i) && __ldg(a.bias + my_i) == __ldg(a.bias + next_i));
        if (!near && __any_sync(FULL_MASK, unsure)) {
            // Mostly the picks and the best of the rest have to be ordered, and what
            // comes after is out of reach of the last place.
            const uint32_t last = __shfl_sync(FULL_MASK, my_key, K - 1);
            if (a.score == MP_SCORE_SIGMOID && K < 32 && !too_near(last, after, err))
                pick = picks_in_order(a, l, lane, K,
                                      lane == K ? (rest != 0u ? static_cast<int>(rest_i) : -1) : pick);
            else
                near = true;
        }
    }
    return __all_sync(FULL_MASK, !near);
}

// KT > 0: a form for K = KT with the rounds unrolled (K = 8, kernels alone: 32,768 x 256,
// sigmoid, bias 32.6 -> 29.7 us, with groups 41.5 -> 40.3, softmax without a bias 29.1 -> 26.2;
// 16,384 x 128 11.3 -> 10.4, raw bf16 11.7 -> 11.3).  Compiled for 4 CTAs per
// SM up to 256 experts (32,768 x 256, sigmoid, bias: 41.4 us with 3, 38.7 with 4
// when this was chosen, 28.7 now), 3 up to 512 (16,383 x 512: 64.5 us with 1, 51.9 with 2,
// 48.7 with 3; 29 now) and 2 up to 1,024 (106.8 with 1, 90.9 with 2; 60 now).
template <typename L, int PER, int KT>
__global__ void __launch_bounds__(RT_THREADS, PER <= 8 ? 4 : PER <= 16 ? 3 : 2) k_route(const RouteArgs a)
{
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * RT_WARPS + (threadIdx.x >> 5);
    if (t >= a.T) return;   // whole warps leave together
    const L *l = static_cast<const L *>(a.logits) + t * a.E;
    float v[PER], b[PER];
    load_token<L, PER>(a, l, lane, v, b);
    int pick;
    if (!choose_fast<L, PER, KT>(a, l, v, b, lane, pick)) pick = choose_exact<L, PER>(a, l, lane);

    // The weights.  sigmoid(v) is exp(v) for v far below zero; where all
    // picks are there, their ratio is taken from exp(v_k - m), which does not
    // underflow.
    const float pv = pick >= 0 ? fminf(logit(l + pick), FLT_MAX) : -INFINITY;
    const float m = pick_max<KT>(pv);
    float s;
    if (a.score == MP_SCORE_SIGMOID && !(a.renorm && m < -40.0f))
        s = pick >= 0 ? __fdiv_rn(1.0f, 1.0f + expf(-pv)) : 0.0f;
    else if (a.score == MP_SCORE_SIGMOID || a.renorm)
        s = pick >= 0 ? expf(pv - m) : 0.0f;
    else {
        float top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int j = 0; j < PER; ++j) top = fmaxf(top, v[j]);
        top = warp_max(top);
#pragma unroll
        for (int j = 0; j < PER; ++j) sum += usable(v[j]) ? expf(v[j] - top) : 0.0f;
        sum = warp_sum(sum);
        s = pick >= 0 ? __fdiv_rn(expf(pv - top), sum) : 0.0f;
    }
    if (a.renorm) s = __fdiv_rn(s, pick_sum<KT>(s));
    if (lane < a.K) {
        a.idx[t * a.K + lane] = pick;
        a.weights[t * a.K + lane] = pick >= 0 ? a.scale * s : 0.0f;
    }
}

struct RouteBwdArgs {
    const float *g_weights;
    const void *logits;
    const int32_t *idx;
    int64_t T;
    int E, K, score, renorm;
    float scale;
    void *g_logits;
};

// renorm: with p the weights before scaling, g_l = scale p_k (g_k - sum_j g_j p_j),
// times 1 - s_k for the sigmoid.  Raw weights: sigmoid scale g_k s_k (1 - s_k);
// softmax scale s_e ([e picked] g_k - sum_j g_j s_j) for every expert.
// VEC: the row is whole chunks of 4 logits, aligned: lane l then holds chunks l,
// l+32, ...; otherwise single ones.
template <typename L, int W> struct alignas(sizeof(L) * W) Chunk {
    L at[W];
};

template <typename L, int PER, bool VEC>
__global__ void __launch_bounds__(RT_THREADS) k_route_bwd(const RouteBwdArgs a)
{
    pdl_trigger();
    pdl_wait();
    constexpr int W = VEC ? 4 : 1, CHUNKS = PER / W;
    typedef Chunk<L, W> C;
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * RT_WARPS + (threadIdx.x >> 5);
    if (t >= a.T) return;
    const L *l = static_cast<const L *>(a.logits) + t * a.E;
    L *gl = static_cast<L *>(a.g_logits) + t * a.E;
    int pick = lane < a.K ? __ldg(a.idx + t * a.K + lane) : -1;
    if (pick >= a.E) pick = -1;
    const float g = pick >= 0 ? a.scale * __ldg(a.g_weights + t * a.K + lane) : 0.0f;
    const float pv = pick >= 0 ? fminf(logit(l + pick), FLT_MAX) : -INFINITY;
    const bool dense = a.score == MP_SCORE_SOFTMAX && !a.renorm;
    float at_pick;
    if (!dense) {
        C zero;
#pragma unroll
        for (int i = 0; i < W; ++i) put(zero.at + i, 0.0f);
        for (int e = lane * W; e < a.E; e += 32 * W) *reinterpret_cast<C *>(gl + e) = zero;
        float left = 1.0f, s;   // 1 - s of the sigmoid
        const float m = warp_max(pv);
        if (a.score == MP_SCORE_SIGMOID) {
            left = __fdiv_rn(1.0f, 1.0f + expf(pv));
            s = (a.renorm && m < -40.0f) ? expf(pv - m) : __fdiv_rn(1.0f, 1.0f + expf(-pv));
        } else {
            s = expf(pv - m);
        }
        if (pick < 0) s = 0.0f;
        if (a.renorm) {
            const float p = __fdiv_rn(s, warp_sum(s));
            const float d = warp_sum(pick >= 0 ? g * p : 0.0f);
            at_pick = p * (g - d) * left;
        } else {
            at_pick = g * s * left;
        }
    } else {
        float v[CHUNKS][W], top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int j = 0; j < CHUNKS; ++j) {
            const int e = (lane + 32 * j) * W;
            C x;
            if (e < a.E) x = *reinterpret_cast<const C *>(l + e);
#pragma unroll
            for (int i = 0; i < W; ++i) {
                v[j][i] = e < a.E ? logit_value(x.at[i]) : -INFINITY;
                v[j][i] = usable(v[j][i]) ? fminf(v[j][i], FLT_MAX) : -INFINITY;
                top = fmaxf(top, v[j][i]);
            }
        }
        top = warp_max(top);
#pragma unroll
        for (int j = 0; j < CHUNKS; ++j)
#pragma unroll
            for (int i = 0; i < W; ++i) {
                v[j][i] = usable(v[j][i]) ? expf(v[j][i] - top) : 0.0f;
                sum += v[j][i];
            }
        sum = warp_sum(sum);
        const float inv = sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
        const float s = pick >= 0 ? expf(pv - top) * inv : 0.0f;
        const float d = warp_sum(pick >= 0 ? g * s : 0.0f);
#pragma unroll
        for (int j = 0; j < CHUNKS; ++j) {
            const int e = (lane + 32 * j) * W;
            C x;
#pragma unroll
            for (int i = 0; i < W; ++i) put(x.at + i, -v[j][i] * inv * d);
            if (e < a.E) *reinterpret_cast<C *>(gl + e) = x;
        }
        at_pick = s * (g - d);
    }
    __syncwarp();   // what is stored above lands before the picks' gradients
    if (pick >= 0) put(gl + pick, at_pick);
}

template <typename L> mp_status_t launch_route(const RouteArgs &a, cudaStream_t s)
{
    const unsigned blocks = static_cast<unsigned>((a.T + RT_WARPS - 1) / RT_WARPS);
    const int per = (a.E + 31) / 32;
    if (per <= 4 && a.K == 8)
        (void)launch_pdl(k_route<L, 4, 8>, blocks, RT_THREADS, 0, s, a);
    else if (per <= 8 && a.K == 8)
        (void)launch_pdl(k_route<L, 8, 8>, blocks, RT_THREADS, 0, s, a);
    else if (per <= 4)
        (void)launch_pdl(k_route<L, 4, 0>, blocks, RT_THREADS, 0, s, a);
    else if (per <= 8)
        (void)launch_pdl(k_route<L, 8, 0>, blocks, RT_THREADS, 0, s, a);
    else if (per <= 16)
        (void)launch_pdl(k_route<L, 16, 0>, blocks, RT_THREADS, 0, s, a);
    else
        (void)launch_pdl(k_route<L, 32, 0>, blocks, RT_THREADS, 0, s, a);
    return check_launch();
}

template <typename L> mp_status_t launch_route_bwd(const RouteBwdArgs &a, cudaStream_t s)
{
    const unsigned blocks = static_cast<unsigned>((a.T + RT_WARPS - 1) / RT_WARPS);
    const int per = (a.E + 31) / 32;
    const uintptr_t both = reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.g_logits);
    const bool vec = a.E % 4 == 0 && both % (4 * sizeof(L)) == 0;
    if (per <= 8 && vec)
        (void)launch_pdl(k_route_bwd<L, 8, true>, blocks, RT_THREADS, 0, s, a);
    else if (per <= 8)
        (void)launch_pdl(k_route_bwd<L, 8, false>, blocks, RT_THREADS, 0, s, a);
    else
        (void)launch_pdl(k_route_bwd<L, 32, false>, blocks, RT_THREADS, 0, s, a);
    return check_launch();
}

mp_status_t route_sizes(int64_t T, int32_t E, int32_t K, int32_t score, int32_t dtype)
{
    if (T < 0 || E < 1 || K < 1 || K > E || score < MP_SCORE_SOFTMAX || score > MP_SCORE_SIGMOID ||
        dtype < MP_DTYPE_BF16 || dtype > MP_DTYPE_FP32)
        return MP_ERR_INVALID_ARG;
    if (E > MP_MAX_EXPERTS || K > 32 || T > INT32_MAX) return MP_ERR_UNSUPPORTED;
    return MP_OK;
}

}  // namespace
}  // namespace mp

using namespace mp;

extern "C" mp_status_t mp_route(const void *logits, int32_t dtype, const float *bias, int64_t T,
                                int32_t E, int32_t K, int32_t score, int32_t n_groups,
                                int32_t topk_groups, int32_t group_top, int32_t renorm,
                                float scale, int32_t *idx, float *weights, mp_stream_t stream)
{
    if (const mp_status_t s = route_sizes(T, E, K, score, dtype); s != MP_OK) return s;
    if (n_groups < 1 || topk_groups < 1 || group_top < 1 || group_top > 2)
        return MP_ERR_INVALID_ARG;
    if (n_groups > 32) return MP_ERR_UNSUPPORTED;
    if (E % n_groups != 0 || topk_groups > n_groups ||
        static_cast<int64_t>(topk_groups) * (E / n_groups) < K)
        return MP_ERR_INVALID_ARG;
    if (T == 0) return MP_OK;
    if (logits == nullptr || idx == nullptr || weights == nullptr) return MP_ERR_INVALID_ARG;
    // Groups of one expert each: the best experts of the best groups are the best experts.
    if (n_groups == E) n_groups = topk_groups = group_top = 1;
    const RouteArgs a = {logits, bias, T, E, K, score, n_groups, topk_groups, group_top, renorm,
                         static_cast<uint32_t>(((1ull << 32) + E / n_groups - 1) / (E / n_groups)),
                         scale, idx, weights};
    const cudaStream_t s = as_stream(stream);
    return dtype == MP_DTYPE_FP32   ? launch_route<float>(a, s)
           : dtype == MP_DTYPE_BF16 ? launch_route<__nv_bfloat16>(a, s)
                                    : launch_route<__half>(a, s);
}

extern "C" mp_status_t mp_route_bwd(const float *g_weights, const void *logits, int32_t dtype,
                                    const int32_t *idx, int64_t T, int32_t E, int32_t K,
                                    int32_t score, int32_t renorm, float scale, void *g_logits,
                                    mp_stream_t stream)
{
    if (const mp_status_t s = route_sizes(T, E, K, score, dtype); s != MP_OK) return s;
    if (T == 0) return MP_OK;
    if (g_weights == nullptr || logits == nullptr || idx == nullptr || g_logits == nullptr)
        return MP_ERR_INVALID_ARG;
    const RouteBwdArgs a = {g_weights, logits, idx, T, E, K, score, renorm, scale, g_logits};
    const cudaStream_t s = as_stream(stream);
    return dtype == MP_DTYPE_FP32   ? launch_route_bwd<float>(a, s)
           : dtype == MP_DTYPE_BF16 ? launch_route_bwd<__nv_bfloat16>(a, s)
                                    : launch_route_bwd<__half>(a, s);
}
