// The end of a group of the norms whose wait for a row's bulk copies was given up, each case a CTA: rows that came,
// rows that are on their way, and slots that take no other.  A row on its way is bytes that its phase still
// asks for; another warp ends them after 20 ms.  Prints for each case whether the group waited for that, whether
// a copy asked for after the wait was started, and the status.
#include <stdio.h>

#include "norm.cuh"

namespace mp {
int sm_count() { return 152; }
void set_last_cuda_error(cudaError_t) {}

constexpr int W = 64, H = 1024;
struct Case {
    int slots, came, coming;   // rows, one after another from slot 0 on
    int left;                  // rows that the loop still goes by, with no copies
};

__global__ void __launch_bounds__(2 * W) k_ring(const Case *cases, const NormInputs in, int32_t *out)
{
    typedef NormGroup<__nv_bfloat16, ROWS_BULK, 2> G;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ volatile int released;
    const Case c = cases[blockIdx.x];
    int32_t *const to = out + 3 * blockIdx.x;
    G g;
    g.begin(smem, W, 2, H);   // the second group is the other warps
    uint8_t *const slots = smem + 4096;
    if (threadIdx.x == 0) {
        released = 0;
        to[2] = 0;
        for (int r = 0; r < c.came + c.coming; ++r) {
            const uint32_t bar = g.bars + 8 * (r % c.slots);
            mbar_expect(bar, 16);
            if (r < c.came)
                asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], 16;" ::"r"(bar) : "memory");
        }
        *g.gave_up = 1;
    }
    for (int i = threadIdx.x; i < 2 * H / 4; i += blockDim.x) reinterpret_cast<uint32_t *>(slots)[i] = 0x5a5a5a5au;
    __syncthreads();
    if (g.group == 0) {
        int at = 0;
        for (int r = 0; r < c.came + c.coming + c.left; ++r) at = g.after(at, c.slots);
        g.fetch<1>(in, 0, 1, slots, 4096, at);
        g.finish(at, c.slots, to + 2);
        if (g.tid == 0) {
            to[0] = released;
            to[1] = reinterpret_cast<volatile uint32_t *>(slots)[0] == 0x5a5a5a5au;
        }
    } else if (g.tid == 0) {
        for (const uint64_t t0 = now_ns(); now_ns() - t0 < 20000000ull;) {
        }
        released = 1;
        __threadfence_block();
        const uint32_t bars = g.bars - NORM_SLOTS * 8;
        for (int r = c.came; r < c.came + c.coming; ++r)
            asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], 16;" ::"r"(bars + 8 * (r % c.slots)) : "memory");
    }
    __syncthreads();
}
}  // namespace mp

using namespace mp;

int main()
{
    Case cases[200];
    int n = 0;
    for (int slots = 1; slots <= 3; ++slots)
        for (int came = 0; came <= 2 * slots; ++came)
            for (int coming = 1; coming <= slots; ++coming)
                for (int left = 0; left <= 2; ++left) cases[n++] = {slots, came, coming, left};
    Case *d_cases;
    int32_t *d_out, out[600];
    void *row;
    if (cudaMalloc(&d_cases, sizeof(cases)) || cudaMalloc(&d_out, sizeof(out)) || cudaMalloc(&row, 2 * H) ||
        cudaMemset(row, 1, 2 * H) || cudaMemcpy(d_cases, cases, sizeof(cases), cudaMemcpyHostToDevice))
        return 2;
    NormInputs in = {};
    for (int i = 1; i < 5; ++i) in.slot[i] = -1;
    in.add(0, {row, 0});
    k_ring<<<n, 2 * W, 4096 + 2 * H>>>(d_cases, in, d_out);
    if (cudaMemcpy(out, d_out, sizeof(int32_t) * 3 * n, cudaMemcpyDeviceToHost)) return 2;
    int wrong = 0;
    for (int i = 0; i < n; ++i)
        if (out[3 * i] != 1 || out[3 * i + 1] != 1 || out[3 * i + 2] != MP_STATUS_STALLED) {
            ++wrong;
            printf("slots %d, came %d, coming %d, left %d: waited %d, nothing copied %d, status %d\n", cases[i].slots,
                   cases[i].came, cases[i].coming, cases[i].left, out[3 * i], out[3 * i + 1], out[3 * i + 2]);
        }
    printf("%d of %d wrong\n", wrong, n);
    return wrong != 0;
}
