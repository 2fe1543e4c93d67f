// How the norms' rows are laid out, checked on the host over sizes and forms: prints a line
// for each plan that would not do.
#include <stdio.h>

#include <vector>

#include "norm.cuh"

namespace mp {
int sm_count() { return 152; }
void set_last_cuda_error(cudaError_t) {}

int wrong = 0;
#define WANT(cond, what)                                                                                             \
    do {                                                                                                             \
        if (!(cond) && ++wrong <= 20)                                                                                \
            printf("%s: H %d, T %lld, %zu bytes, form %d, tensors %d, held %d, sums %d: W %d, R %d, slots %d\n", what, \
                   H, static_cast<long long>(T), sizeof(D), form, tensors, held, sums, p.W, p.R, p.stages);          \
    } while (0)

// Whether the W threads of a row have each of its columns once.
template <typename D, int M, int C> bool covers(int W, int H)
{
    std::vector<int> times(H, 0);
    for (int tid = 0; tid < W; ++tid) {
        NormGroup<D, M, C> g;
        g.W = W;
        g.H = H;
        g.tid = tid;
        for (int i = 0; i < g.N2; ++i)
            for (const int c : {g.col(i), g.col(i) + g.beside()})
                if (c < H) ++times[c];
    }
    for (const int n : times)
        if (n != 1) return false;
    return true;
}

template <typename D> void check(int H, int64_t T, bool vec, int tensors, int held, int sums, bool forward, bool columns)
{
    const int form = H > 16 * NORM_THREADS ? (vec ? ROWS_VEC : ROWS_ANY)
                     : vec                 ? (norm_by_bulk<D>(H) ? ROWS_BULK : ROWS_VEC)
                                           : (norm_is_narrow(H) ? ROWS_NARROW : ROWS_ANY);
    bool staged = H <= 16 * NORM_THREADS;
    NormPlan p = norm_plan<D>(T, H, staged ? 2 : 4, staged ? NORM_THREADS : 2 * NORM_THREADS, form, tensors, held, sums, forward);
    if (staged && p.stages < 1) {   // the unstaged form in its place
        WANT(!forward && !norm_is_narrow(H), "unstaged");
        if (forward) return;
        staged = false;
        p = norm_plan<D>(T, H, 4, 2 * NORM_THREADS, vec ? ROWS_VEC : ROWS_ANY, tensors, held, sums, forward);
    }
    WANT(p.W * p.R % 32 == 0, "no whole warps");
    WANT(p.W * p.R <= (staged ? 1 : 2) * NORM_THREADS, "threads");
    WANT(p.smem <= static_cast<size_t>(NORM_MOST), "shared memory");
    if (staged) {
        const int piles = p.W < 32 ? p.W * p.R / 32 : p.R;
        WANT(forward || static_cast<int64_t>(piles) * norm_wide(H) * 4 <= static_cast<int64_t>(p.R) * p.stages * tensors * p.pitch,
             "sums of the groups do not fit the slots");
    }
    if (!columns || (T != 1 && T != 1 << 30)) return;   // a row's threads do not go by T
    const bool ok = !staged ? (vec ? covers<D, ROWS_VEC, 4>(p.W, H) : covers<D, ROWS_ANY, 4>(p.W, H))
                    : form == ROWS_NARROW ? covers<D, ROWS_NARROW, 2>(p.W, H)
                    : form == ROWS_ANY    ? covers<D, ROWS_ANY, 2>(p.W, H)
                                          : covers<D, ROWS_VEC, 2>(p.W, H);
    WANT(ok, "columns");
}

template <typename D> void sweep()
{
    for (int H = 1; H <= MP_MAX_NORM_WIDTH; H += H < 320 || (H > 8150 && H < 8200) ? 1 : H < 8200 ? 13 : 1021)
        for (const int64_t T : {1ll, 2ll, 31ll, 153ll, 1000ll, 2433ll, 5000ll, 10000ll, 20000ll, 40000ll, 1ll << 30})
            for (int vec = 0; vec < (H * sizeof(D) % 16 == 0 ? 2 : 1); ++vec)
                for (int norms = 1; norms <= 3; ++norms)
                    for (int gate = MP_GATE_NONE; gate <= MP_GATE_ELEMENT; ++gate) {
                        const bool post = norms & 1, pre = norms & 2, channel = gate == MP_GATE_CHANNEL, element = gate == MP_GATE_ELEMENT;
                        for (int b = 0; b <= post + pre; ++b)          // biases
                            for (int residual = 0; residual <= 1; ++residual)
                                check<D>(H, T, vec, 1 + residual + element, post + pre + b + channel, 0, true, b == post + pre);
                        for (int post_b = 0; post_b <= post; ++post_b)
                            for (int sums = 0; sums <= post + pre + channel; ++sums)
                                for (int g_s = !pre; g_s <= 1; ++g_s)
                                    check<D>(H, T, vec, g_s + 2 * pre + (post || gate != MP_GATE_NONE) + element,
                                             post + pre + post_b + channel, sums, false, sums == 0 || sums == post + pre + channel);
                    }
}
}  // namespace mp

int main()
{
    mp::sweep<float>();
    mp::sweep<__half>();
    mp::sweep<__nv_bfloat16>();
    printf("%d wrong\n", mp::wrong);
    return mp::wrong != 0;
}
