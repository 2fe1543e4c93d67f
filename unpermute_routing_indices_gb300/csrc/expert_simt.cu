// The experts' products on the ordinary arithmetic units, for any width and
// alignment.
//
// Each CTA computes a 64 x 64 tile of one expert's product, 4 x 4 results per
// thread, from 16-deep slices of both operands held as fp32 in shared memory;
// operands are addressed by strides, so one kernel serves x w^T, g w and g^T x.
// The finished tile goes through shared memory to the epilogue, which works on
// 32 columns of a row per thread.
#include "expert.cuh"

namespace mp {
namespace {

constexpr int ST = 64, SD = 16, SIMT_THREADS = 256;

__device__ __forceinline__ float bf16_at(const mp_bf16_t *p)
{
    return __uint_as_float(static_cast<uint32_t>(__ldg(p)) << 16);
}

template <int MODE, bool GATED>
__global__ void __launch_bounds__(SIMT_THREADS) k_expert_simt(const ExpertCall c)
{
    pdl_trigger();
    pdl_wait();
    __shared__ int start[MP_MAX_EXPERTS + 1], tiles[MP_MAX_EXPERTS + 1];
    __shared__ float sa[SD][ST + 4], sb[GATED ? 2 : 1][SD][ST + 4];
    float(*sc)[ST + 1] = reinterpret_cast<float(*)[ST + 1]>(&sa[0][0]);   // one row strip at a time
    static_assert(sizeof(sa) >= 16 * (ST + 1) * sizeof(float), "a strip of 16 rows fits");

    if (threadIdx.x < 32)
        expert_starts(c.offsets, c.E, c.R, ST, threadIdx.x, start, tiles,
                      blockIdx.x + blockIdx.y + blockIdx.z == 0 ? c.status : nullptr);
    __syncthreads();

    if (MODE != WGRAD && c.epi.zero_rest) {
        const int64_t blocks = static_cast<int64_t>(gridDim.x) * gridDim.y;
        zero_rest(c.epi, start[c.E], c.R,
                  (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * SIMT_THREADS + threadIdx.x,
                  blocks * SIMT_THREADS);
    }

    // Rows m0..m1 of A, columns from n0 of B, contraction over [0,depth).
    int e, m0, m1, depth;
    int64_t sam, sak, sbn, sbk;
    const mp_bf16_t *a = c.a, *b = c.b;
    if (MODE == WGRAD) {
        e = blockIdx.z;
        m0 = blockIdx.x * ST;
        m1 = c.N;
        depth = start[e + 1] - start[e];
        a += static_cast<int64_t>(start[e]) * c.N;
        b += static_cast<int64_t>(start[e]) * c.K;
        sam = 1; sak = c.N; sbn = 1; sbk = c.K;
    } else {
        if (static_cast<int>(blockIdx.x) >= tiles[c.E]) return;
        e = expert_of_tile(tiles, c.E, blockIdx.x);
        m0 = start[e] + (blockIdx.x - tiles[e]) * ST;
        m1 = start[e + 1];
        b += static_cast<int64_t>(e) * c.N * c.K;
        if (MODE == FWD) {
            depth = c.K;
            sam = c.K; sak = 1; sbn = c.K; sbk = 1;
        } else {
            depth = c.N;
            sam = c.N; sak = 1; sbn = 1; sbk = c.K;
        }
    }
    const int n0 = blockIdx.y * ST, cols = c.epi.cols;
    const int64_t part_b = static_cast<int64_t>(cols) * sbn;   // GATED: from the gate to the others

    float acc[GATED ? 2 : 1][4][4] = {};
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int k0 = 0; k0 < depth; k0 += SD) {
        for (int i = threadIdx.x; i < SD * ST; i += SIMT_THREADS) {
            // The index that runs fastest follows the operand's unit stride.
            const int ka = sak == 1 ? i % SD : i / ST, ma = sak == 1 ? i / SD : i % ST;
            sa[ka][ma] = (k0 + ka < depth && m0 + ma < m1)
                             ? bf16_at(a + (m0 + ma) * sam + (k0 + ka) * sak) : 0.0f;
            const int kb = sbk == 1 ? i % SD : i / ST, nb = sbk == 1 ? i / SD : i % ST;
            const bool in = k0 + kb < depth && n0 + nb < cols;
            const mp_bf16_t *q = b + (n0 + nb) * sbn + (k0 + kb) * sbk;
            sb[0][kb][nb] = in ? bf16_at(q) : 0.0f;
            if (GATED) sb[1][kb][nb] = in ? bf16_at(q + part_b) : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < SD; ++k) {
            float fa[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) fa[i] = sa[k][ty * 4 + i];
#pragma unroll
            for (int g = 0; g < (GATED ? 2 : 1); ++g)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float fb = sb[g][k][tx + 16 * j];
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[g][i][j] = fmaf(fa[i], fb, acc[g][i][j]);
                }
        }
        __syncthreads();
    }

    // 16 rows at a time: the strip of the gate, then of the others.
    for (int strip = 0; strip < ST / 16; ++strip) {
        float z[EPI_COLS], u[EPI_COLS];
        const int r = threadIdx.x >> 1, cc = (threadIdx.x & 1) * EPI_COLS;
#pragma unroll
        for (int g = 0; g < (GATED ? 2 : 1); ++g) {
            if (ty / 4 == strip) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) sc[(ty & 3) * 4 + i][tx + 16 * j] = acc[g][i][j];
            }
            __syncthreads();
            if (r < 16) {
#pragma unroll
                for (int i = 0; i < EPI_COLS; ++i) (g == 0 ? z : u)[i] = sc[r][cc + i];
            }
            __syncthreads();
        }
        const int row = m0 + strip * 16 + r, col = n0 + cc;
        if (r < 16 && row < m1 && col < cols) {
            const int n = min(EPI_COLS, cols - col);
            RowWriter w;
            if (MODE == FWD) epi_fwd<GATED>(c.epi, w, e, row, col, n, true, z, u);
            if (MODE == DGRAD) epi_dgrad(c.epi, w, row, col, n, true, z);
            if (MODE == WGRAD)
                epi_wgrad(c.epi, w, static_cast<int64_t>(e) * c.N + row, col, n, true, z);
        }
    }
}

}  // namespace

template <int MODE> mp_status_t expert_simt(const ExpertCall &c)
{
    const unsigned ny = (c.epi.cols + ST - 1) / ST;
    if (ny > 65535) return MP_ERR_UNSUPPORTED;
    const dim3 grid = MODE == WGRAD ? dim3((c.N + ST - 1) / ST, ny, c.E)
                                    : dim3(c.R / ST + min(c.E, c.R), ny);
    if (MODE == FWD && act_gated(c.epi.act))
        (void)launch_pdl(k_expert_simt<MODE, MODE == FWD>, grid, SIMT_THREADS, 0, c.stream, c);
    else
        (void)launch_pdl(k_expert_simt<MODE, false>, grid, SIMT_THREADS, 0, c.stream, c);
    return check_launch();
}

template mp_status_t expert_simt<FWD>(const ExpertCall &);
template mp_status_t expert_simt<DGRAD>(const ExpertCall &);
template mp_status_t expert_simt<WGRAD>(const ExpertCall &);

}  // namespace mp
