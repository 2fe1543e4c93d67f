// mp_expert_gemm for experts with few rows: answering single tokens.
//
// The weights' bytes bound it, so the tile is turned: 128 rows of w[e] (and the
// 128 of the other half when gated) against up to 32 rows of x, and what counts
// is that every SM keeps loads in flight.  Warp 0 streams the weights by TMA, warp 1
// issues the products (accumulator: a weight row per lane, a row of x per
// column), warps 2-5 run the epilogue, whose stores are 32 neighbouring columns of
// a row.  Two CTAs share an SM, so that one's epilogue or start covers the other.
// With enough tiles the CTAs are persistent (SPLIT 1).  With fewer, the
// contraction of a tile is split over the SPLIT CTAs of a cluster; each leaves its
// partial sums in its shared memory, and they are added in rank order through
// distributed shared memory, so a result does not depend on timing.
#include "expert.cuh"
#include "tc.cuh"

namespace mp {
namespace {

constexpr int FM = 128, FT = 32, FK = 64;   // weight rows, rows of x, depth of a slice
constexpr int FEW_THREADS = 192;
constexpr int W_BYTES = FM * FK * 2, X_BYTES = FT * FK * 2;

template <bool GATED> struct Few {
    static constexpr int PARTS = GATED ? 2 : 1;
    static constexpr int STAGES = GATED ? 3 : 5;
    static constexpr int STAGE = PARTS * W_BYTES + X_BYTES;
    static constexpr int COLS = 2 * PARTS * FT;   // TMEM columns: two accumulators
    struct Shared {
        uint64_t full[STAGES], empty[STAGES], acc_full[2], acc_empty[2], drained;
        uint32_t tmem;
        int gave_up;
    };
    // With the experts' tables of E + 1 entries each.
    static constexpr size_t smem(int E) { return 1024 + STAGES * STAGE + sizeof(Shared) + 8 * (E + 1); }
};
// Two CTAs on an SM (233,472 bytes, 1,024 of them reserved for each): gated up to
// 481 experts, otherwise any number.
constexpr size_t HALF_SM = 233472 / 2 - 1024;
static_assert(Few<true>::smem(480) <= HALF_SM && Few<false>::smem(MP_MAX_EXPERTS) <= HALF_SM, "two CTAs on an SM");
static_assert(2 * FM * FT * 4 <= Few<true>::STAGES * Few<true>::STAGE, "partial sums fit the ring");

__device__ __forceinline__ float peer_value(uint32_t addr, uint32_t rank)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at_rank(addr, rank)) : "memory");
    return v;
}

// The epilogue of one row of x at 32 columns, one a lane.
template <bool GATED>
__device__ __forceinline__ void lane_epilogue(const ExpertEpi &p, int64_t row, int col, int lane,
                                              float bz, float bu, float residual, float z, float u)
{
    const bool in = col < p.cols;
    constexpr int parts = GATED ? 2 : 1;
    z += bz;
    if (GATED) u += bu;
    if (p.save != MP_SAVE_NONE) {
#pragma unroll
        for (int q = 0; q < parts; ++q) {
            const float v = q == 0 ? z : u;
            const int64_t at = (row * parts + q) * p.cols + col;
            if (p.save == MP_SAVE_BF16) {
                const float f[1] = {v};
                if (in) static_cast<mp_bf16_t *>(p.z)[at] = pack(f);
            } else {
                const float zf = finite_or_nan(v), mag = in ? fmaxf(fabsf(zf), 0.0f) : 0.0f;
                const int x = ckpt_exponent(__uint_as_float(__reduce_max_sync(FULL_MASK, __float_as_uint(mag))));
                if (in) static_cast<uint8_t *>(p.z)[at] = static_cast<uint8_t>(e4m3x4(zf * pow2_biased(254 - x), 0, 0, 0));
                if (lane == 0 && in)
                    p.z_exp[(row * parts + q) * ckpt_blocks(p.cols) + col / EPI_COLS] = static_cast<uint8_t>(x);
            }
        }
    }
    switch (act_inner(p.act)) {
    case MP_ACT_SILU: z = act_value<MP_ACT_SILU>(z); break;
    case MP_ACT_GELU: z = act_value<MP_ACT_GELU>(z); break;
    case MP_ACT_RELU: z = act_value<MP_ACT_RELU>(z); break;
    default: break;
    }
    if (GATED) z *= u;
    const float f[1] = {z + residual};
    if (in) p.out[row * p.cols + col] = pack(f);
}

__device__ __forceinline__ float bf16_or_zero(const mp_bf16_t *p, bool in)
{
    float f[1] = {0.0f};
    if (in) unpack(ld_stream(p), f);
    return f[0];
}

template <bool GATED>
__global__ void __launch_bounds__(FEW_THREADS, 2)
    k_expert_few(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                 const ExpertCall c, int split)
{
    typedef Few<GATED> L;
    constexpr int PARTS = L::PARTS, STAGES = L::STAGES;
    extern __shared__ uint8_t raw[];
    uint8_t *ring = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    typename L::Shared &s = *reinterpret_cast<typename L::Shared *>(ring + STAGES * L::STAGE);
    int *const start = reinterpret_cast<int *>(&s + 1), *const tiles = start + c.E + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int *gave_up = &s.gave_up;

    if (threadIdx.x == 0) {
        tma_prefetch(&map_w);
        tma_prefetch(&map_x);
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(smem_u32(&s.full[i]), 1);
            mbar_init(smem_u32(&s.empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&s.acc_full[i]), 1);
            mbar_init(smem_u32(&s.acc_empty[i]), 4);
        }
        mbar_init(smem_u32(&s.drained), 1);
        mbar_init_fence();
        s.gave_up = 0;
    }
    if (warp == 1) tmem_alloc(smem_u32(&s.tmem), L::COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_trigger();   // only with the TMEM in hand (see k_expert_tc)
    pdl_wait();
    if (warp == 0)
        expert_starts(c.offsets, c.E, c.R, FT, lane, start, tiles,
                      blockIdx.x == 0 ? c.status : nullptr);
    __syncthreads();

    const uint32_t tmem = s.tmem;
    const int cols = c.epi.cols, nt = (cols + FM - 1) / FM;
    const int64_t total = static_cast<int64_t>(tiles[c.E]) * nt;
    const int rank = split > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int64_t first = blockIdx.x / split, step = gridDim.x / split;
    // This CTA's slices of the contraction.
    const int slices = (c.K + FK - 1) / FK;
    const int k0 = slices * rank / split, k1 = slices * (rank + 1) / split;
    constexpr uint32_t idesc = mma_desc(FM, FT, false, false);

    // Tile t: column block by column block of an expert, its row blocks next to
    // each other, so that they share the weights in L2.
    const auto tile = [&](int64_t t, int &e, int &col, int &row, int &rows) {
        e = expert_of_tile(tiles, c.E, static_cast<int>(t / nt));
        const int mt = tiles[e + 1] - tiles[e];
        const int64_t at = t - static_cast<int64_t>(tiles[e]) * nt;
        col = static_cast<int>(at / mt) * FM;
        row = start[e] + static_cast<int>(at % mt) * FT;
        rows = min(start[e + 1] - row, FT);
    };

    if (warp == 0) {
        if (lane == 0) {
            uint32_t n = 0;
            for (int64_t t = first; t < total && !*gave_up; t += step) {
                int e, col, row, rows;
                tile(t, e, col, row, rows);
                for (int k = k0; k < k1; ++k, ++n) {
                    const int i = n % STAGES;
                    if (!mbar_wait(smem_u32(&s.empty[i]), ((n / STAGES) & 1) ^ 1, gave_up)) break;
                    const uint32_t bar = smem_u32(&s.full[i]), a = smem_u32(ring + i * L::STAGE);
                    mbar_expect(bar, L::STAGE);
                    for (int q = 0; q < PARTS; ++q)
                        tma_load(a + q * W_BYTES, &map_w, bar, k * FK, col + q * cols, e);
                    tma_load(a + PARTS * W_BYTES, &map_x, bar, k * FK, row);
                }
            }
            if (*gave_up)
                for (uint32_t q = n > STAGES ? n - STAGES : 0; q < n; ++q)
                    mbar_drain(smem_u32(&s.full[q % STAGES]), (q / STAGES) & 1);
        }
    } else if (warp == 1) {
        uint32_t n = 0, it = 0;
        bool ok = true;
        for (int64_t t = first; t < total && ok; t += step, ++it) {
            const int acc = it & 1;
            ok = __all_sync(FULL_MASK, mbar_wait(smem_u32(&s.acc_empty[acc]), ((it >> 1) & 1) ^ 1, gave_up));
            if (!ok) break;
            tc_fence_after();
            for (int k = k0; k < k1; ++k, ++n) {
                const int i = n % STAGES;
                ok = __all_sync(FULL_MASK, mbar_wait(smem_u32(&s.full[i]), (n / STAGES) & 1, gave_up));
                if (!ok) break;
                tc_fence_after();
                if (lane == 0) {
                    const uint32_t a = smem_u32(ring + i * L::STAGE), x = a + PARTS * W_BYTES;
                    for (int q = 0; q < FK / 16; ++q)
                        for (int h = 0; h < PARTS; ++h)
                            tc_mma(tmem + (acc * PARTS + h) * FT, tile_desc(a + h * W_BYTES + q * 32, 0),
                                   tile_desc(x + q * 32, 0), idesc, k != k0 || q != 0);
                    tc_commit(smem_u32(&s.empty[i]));
                }
                __syncwarp();
            }
            if (ok && lane == 0) tc_commit(smem_u32(&s.acc_full[acc]));
            __syncwarp();
        }
        if (!ok && lane == 0) {
            tc_commit(smem_u32(&s.drained));
            mbar_drain(smem_u32(&s.drained), 0);
            or_status(c.status, MP_STATUS_STALLED);
        }
    } else {
        const int quad = warp & 3;
        if (c.epi.zero_rest)
            zero_rest(c.epi, start[0], start[c.E], c.R, blockIdx.x * 128 + threadIdx.x - 64,
                      static_cast<int64_t>(gridDim.x) * 128);
        uint32_t it = 0;
        for (int64_t t = first; t < total; t += step, ++it) {
            int e, col, row, rows;
            tile(t, e, col, row, rows);
            const int acc = it & 1;
            const int f = col + quad * 32 + lane;   // this lane's column of the result
            // What the epilogue reads is on its way before the sums are there.
            float bz = 0.0f, bu = 0.0f, residual[FT];
            if (split == 1) {
                const mp_bf16_t *bias = c.epi.bias + static_cast<int64_t>(e) * PARTS * cols + f;
                bz = bf16_or_zero(bias, c.epi.bias != nullptr && f < cols);
                if (GATED) bu = bf16_or_zero(bias + cols, c.epi.bias != nullptr && f < cols);
#pragma unroll
                for (int i = 0; i < FT; ++i)
                    residual[i] = bf16_or_zero(c.epi.residual + static_cast<int64_t>(row + i) * cols + f,
                                                     c.epi.residual != nullptr && i < rows && f < cols);
            }
            if (!__all_sync(FULL_MASK, mbar_wait(smem_u32(&s.acc_full[acc]), (it >> 1) & 1, gave_up))) break;
            tc_fence_after();
            const uint32_t d = tmem + acc * PARTS * FT + (static_cast<uint32_t>(quad * 32) << 16);
            float z[FT], u[FT];
            tmem_load32(d, z);
            if (GATED) tmem_load32(d + FT, u);
            tmem_load_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&s.acc_empty[acc]));
            if (split == 1) {
#pragma unroll
                for (int i = 0; i < FT; ++i)
                    if (i < rows) lane_epilogue<GATED>(c.epi, row + i, f, lane, bz, bu, residual[i], z[i], GATED ? u[i] : 0.0f);
            } else {
                float *part = reinterpret_cast<float *>(ring) + quad * 32 + lane;
#pragma unroll
                for (int i = 0; i < FT; ++i)
                    if (i < rows) {
                        part[i * FM] = z[i];
                        if (GATED) part[(FT + i) * FM] = u[i];
                    }
            }
        }
    }
    __syncwarp();
    if (split > 1) {   // one tile a cluster
        cluster_sync();
        if (first < total && warp >= 2) {
            int e, col, row, rows;
            tile(first, e, col, row, rows);
            // Row i's 32 columns of quarter q go to rank (4 i + q) % split.
            for (int w = (warp - 2) * split + rank; w < 4 * rows; w += 4 * split) {
                const int i = w >> 2, q = w & 3, f = col + q * 32 + lane;
                const uint32_t at = smem_u32(ring) + (i * FM + q * 32 + lane) * 4;
                const mp_bf16_t *bias = c.epi.bias + static_cast<int64_t>(e) * PARTS * cols + f;
                const float bz = bf16_or_zero(bias, c.epi.bias != nullptr && f < cols);
                const float bu = GATED ? bf16_or_zero(bias + cols, c.epi.bias != nullptr && f < cols) : 0.0f;
                const float residual = bf16_or_zero(c.epi.residual + static_cast<int64_t>(row + i) * cols + f,
                                                          c.epi.residual != nullptr && f < cols);
                float z = 0.0f, u = 0.0f;
                for (int r = 0; r < split; ++r) {
                    z += peer_value(at, r);
                    if (GATED) u += peer_value(at + FT * FM * 4, r);
                }
                lane_epilogue<GATED>(c.epi, row + i, f, lane, bz, bu, residual, z, u);
            }
        }
        __syncwarp();
        cluster_sync();   // peers have read this CTA's sums
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_free(tmem, L::COLS);
    }
}

template <bool GATED>
mp_status_t launch_few(const ExpertCall &c, const CUtensorMap &w, const CUtensorMap &x)
{
    typedef Few<GATED> L;
    static std::atomic<uint64_t> allowed{0};
    if (!allow_smem(k_expert_few<GATED>, allowed, L::smem(MP_MAX_EXPERTS))) return MP_ERR_CUDA;
    // The most tiles that any offsets give, and CTAs that the SMs hold at once.
    const int64_t most = static_cast<int64_t>(c.R / FT + (c.R < c.E ? c.R : c.E)) * ((c.epi.cols + FM - 1) / FM);
    const int64_t room = (L::smem(c.E) <= HALF_SM ? 2 : 1) * sm_count();
    int split = 1;
    while (split < 8 && most * split * 2 <= room && c.K / FK >= 4 * split) split *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = static_cast<unsigned>(split > 1 ? most * split : most < room ? most : room);
    cfg.blockDim = FEW_THREADS;
    cfg.dynamicSmemBytes = L::smem(c.E);
    cfg.stream = c.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = split > 1 ? 2 : 1;
    (void)cudaLaunchKernelEx(&cfg, k_expert_few<GATED>, w, x, c, split);
    return check_launch();
}

}  // namespace

// Up to 2 rows an expert, 4 when gated (the tile then has twice the weights to a
// row of x), and up to 64 rows in all.  us here / by k_expert_tc: 32 experts of 1,024 x 512,
// 64 rows 9.1 / 10.6, 128 rows 9.5 / 9.0; gated 128 rows 9.3 / 9.0, 528 x 2,048 14.5 / 16.2, 256
// rows 11.5 / 9.0; 128 experts of 4,096 x 2,048, 8 rows 26 / 36; 4 of 1,024 x 1,024, 16 rows 6.0 /
// 9.0, 64 rows 7.7 / 8.9; one of 512 x 512, 16 rows 6.2 / 6.1, 64 rows 7.8 / 6.2.
bool expert_few_takes(const ExpertCall &c)
{
    return expert_by_tma(c, FWD) && (c.R <= 64 || c.R <= (act_gated(c.epi.act) ? 4 : 2) * static_cast<int64_t>(c.E));
}

mp_status_t expert_few(const ExpertCall &c)
{
    CUtensorMap w, x;
    const uint64_t dw[3] = {static_cast<uint64_t>(c.K), static_cast<uint64_t>(c.N), static_cast<uint64_t>(c.E)};
    const uint64_t dx[2] = {static_cast<uint64_t>(c.K), static_cast<uint64_t>(c.R)};
    const uint32_t box_w[3] = {FK, FM, 1}, box_x[2] = {FK, FT};
    if (!make_map(&w, c.b, 3, dw, box_w) || !make_map(&x, c.a, 2, dx, box_x)) {
        set_last_cuda_error(cudaErrorInvalidValue);
        return MP_ERR_CUDA;
    }
    return act_gated(c.epi.act) ? launch_few<true>(c, w, x) : launch_few<false>(c, w, x);
}

}  // namespace mp
