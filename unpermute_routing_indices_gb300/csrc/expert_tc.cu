// The experts' products on the tensor cores.
//
// One persistent kernel for the three products, a CTA per SM.  A tile is 128
// rows by 256 columns (128 gate and 128 other columns when gated) of one expert:
//   FWD    rows of x by rows of w[e], contraction along both rows
//   DGRAD  rows of g along, w[e] across (its columns are the result's)
//   WGRAD  g and x both across: the contraction is over the expert's rows
// Warp 0 loads 64-deep slices of both operands by TMA into a ring, warp 1 issues
// the products into one of two TMEM accumulators, and warps 2-9 take the other
// one through the epilogue, 32 columns of a row per thread and step.  Every CTA derives
// the tiles from the offsets on the device, so that the grid depends on the
// sizes alone and the call can be captured.
// Rows of a tile past the expert's end belong to the next expert: they are
// computed and dropped (FWD, DGRAD).  In WGRAD, where they would enter the sums,
// the last slice's rows up to the next 16 are overwritten with zeros in shared
// memory, whatever they held.
#include "expert.cuh"
#include "tc.cuh"

namespace mp {

int sm_count()
{
    static std::atomic<int> known[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 1;
    if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 1;
    if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

bool make_map(CUtensorMap *m, const void *base, int rank, const uint64_t *dims, const uint32_t *box)
{
    typedef CUresult (*Encode)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                               const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                               const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                               CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static Encode encode = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                             &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<Encode>(f);
    }();
    if (encode == nullptr) return false;
    cuuint64_t d[3], strides[2];
    cuuint32_t b[3], one[3] = {1, 1, 1};
    uint64_t bytes = 2;
    for (int i = 0; i < rank; ++i) {
        d[i] = dims[i];
        b[i] = box[i];
        bytes *= dims[i];
        if (i + 1 < rank) strides[i] = bytes;
    }
    for (int attempt = 0;; ++attempt) {
        if (encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(base), d, strides,
                   b, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   box[0] == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS)
            return true;
        // A thread that has made no runtime call yet (autograd's) has no
        // current context: setting its device gives it one.
        int dev = 0;
        if (attempt > 0 || cudaGetDevice(&dev) != cudaSuccess || cudaSetDevice(dev) != cudaSuccess)
            return false;
    }
}

namespace {

constexpr int BM = 128, BN = 256, BK = 64;
constexpr int STAGES = 4;
constexpr int EPI_WARPS = 8;   // two for each quarter of the accumulator's lanes
constexpr int TC_THREADS = 64 + 32 * EPI_WARPS;
constexpr int A_BYTES = BM * BK * 2, B_BYTES = BN * BK * 2, STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int BOX_BYTES = 64 * 64 * 2;   // a box of 64 rows
constexpr int TMEM_COLS = 2 * BN;

constexpr int STAGING = 32 * EPI_COLS * 2;   // bytes of one warp's tile on its way out

struct TcShared {
    uint64_t full[STAGES], empty[STAGES], acc_full[2], acc_empty[2], drained;
    uint32_t tmem;
    int gave_up;
    int start[MP_MAX_EXPERTS + 1], tiles[MP_MAX_EXPERTS + 1];
};
constexpr size_t TC_SMEM = 1024 + STAGES * STAGE_BYTES + EPI_WARPS * STAGING + sizeof(TcShared);
static_assert(TC_SMEM <= 232448, "shared memory of one SM");

struct Tile {
    int e, m0, m1, c0, row0, depth;   // rows [m0,m1) of the result (of g's columns in WGRAD)
};

template <int MODE>
__device__ __forceinline__ Tile tile_at(const ExpertCall &c, const int *start, const int *tiles,
                                        int64_t t, int nt, int tile_cols)
{
    Tile r;
    if (MODE == WGRAD) {
        const int mt = (c.N + BM - 1) / BM;
        const int64_t per = static_cast<int64_t>(mt) * nt;
        r.e = static_cast<int>(t / per);
        const int64_t at = t - r.e * per;
        r.m0 = static_cast<int>(at % mt) * BM;
        r.m1 = c.N;
        r.c0 = static_cast<int>(at / mt) * tile_cols;
        r.row0 = start[r.e];
        r.depth = start[r.e + 1] - r.row0;
    } else {
        r.e = expert_of_tile(tiles, c.E, static_cast<int>(t / nt));
        const int mt = tiles[r.e + 1] - tiles[r.e];
        const int64_t at = t - static_cast<int64_t>(tiles[r.e]) * nt;
        r.m0 = start[r.e] + static_cast<int>(at % mt) * BM;
        r.m1 = start[r.e + 1];
        r.c0 = static_cast<int>(at / mt) * tile_cols;
        r.row0 = 0;
        r.depth = MODE == FWD ? c.K : c.N;
    }
    return r;
}

// Maps the epilogue stores by, and whether it may (alignment): TO_OUT, TO_SECOND.
struct StoreMaps {
    CUtensorMap map[2];
    bool use[2];
};

// Writes the 32 x 32 tile of a warp (a row per lane) through shared memory: a row
// per lane straight to global memory would touch 32 lines with each store, which
// bounded the weight gradient of many small experts (277 us against 233 on 256
// experts of 128 rows, 1,024 x 2,048).  A full tile leaves by TMA; one with
// fewer rows or columns, or rows that TMA cannot address, by stores of
// neighbouring lanes to neighbouring bytes.  16-byte pieces are placed as TMA's
// 64-byte swizzle has them, which also spreads them over the banks.
struct WarpWriter {
    uint8_t *tile;
    const StoreMaps &maps;
    int lane, rows;   // rows of the 32 that exist

    __device__ __forceinline__ void put(mp_bf16_t *base, int64_t pitch, int which, int64_t row,
                                        int64_t c, int n, bool, const float (&f)[EPI_COLS])
    {
        if (lane == 0) tma_store_read();   // the tile before this one has left
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 4; ++q)
            *reinterpret_cast<uint4 *>(tile + lane * 64 + ((q ^ ((lane >> 1) & 3)) * 16)) = pack8(f + 8 * q);
        const int64_t row0 = __shfl_sync(FULL_MASK, row, 0);
        if (rows == 32 && n == EPI_COLS && maps.use[which]) {
            fence_async_smem();
            __syncwarp();
            if (lane == 0)
                tma_store(&maps.map[which], smem_u32(tile), static_cast<int>(c), static_cast<int>(row0));
            return;
        }
        __syncwarp();
        mp_bf16_t *to = base + row0 * pitch + c;
        if (n == EPI_COLS && maps.use[which]) {
            for (int r = lane >> 2; r < rows; r += 8)
                *reinterpret_cast<uint4 *>(to + r * pitch + (lane & 3) * 8) = *reinterpret_cast<const uint4 *>(
                    tile + r * 64 + (((lane & 3) ^ ((r >> 1) & 3)) * 16));
        } else if (lane < n) {
            for (int r = 0; r < rows; ++r)
                to[r * pitch + lane] = *reinterpret_cast<const uint16_t *>(
                    tile + r * 64 + (((lane >> 3) ^ ((r >> 1) & 3)) * 16) + (lane & 7) * 2);
        }
    }
};

// Brings what the epilogue of columns [c0,c1) of a row will read into L2 while the
// accumulator fills.
__device__ __forceinline__ void prefetch_l2(const void *p, int bytes)
{
    for (int i = 0; i < bytes; i += 128)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char *>(p) + i));
}
template <int MODE>
__device__ __forceinline__ void epi_prefetch(const ExpertEpi &p, int64_t row, int c0, int c1)
{
    if (MODE == FWD) {
        if (p.residual != nullptr) prefetch_l2(p.residual + row * p.cols + c0, 2 * (c1 - c0));
    } else if (p.act != MP_ACT_NONE) {
        const int parts = act_gated(p.act) ? 2 : 1, size = p.save == MP_SAVE_BF16 ? 2 : 1;
        for (int q = 0; q < parts; ++q)
            prefetch_l2(static_cast<const char *>(p.z) + ((row * parts + q) * p.cols + c0) * size,
                        size * (c1 - c0));
    }
}

template <int MODE, bool GATED>
__global__ void __launch_bounds__(TC_THREADS, 1)
    k_expert_tc(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                const __grid_constant__ StoreMaps stores, const ExpertCall c)
{
    extern __shared__ uint8_t raw[];
    uint8_t *ring = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    TcShared &s = *reinterpret_cast<TcShared *>(ring + STAGES * STAGE_BYTES + EPI_WARPS * STAGING);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int *gave_up = &s.gave_up;

    if (threadIdx.x == 0) {
        tma_prefetch(&map_a);
        tma_prefetch(&map_b);
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(smem_u32(&s.full[i]), 1);
            mbar_init(smem_u32(&s.empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&s.acc_full[i]), 1);
            mbar_init(smem_u32(&s.acc_empty[i]), EPI_WARPS);
        }
        mbar_init(smem_u32(&s.drained), 1);
        mbar_init_fence();
        s.gave_up = 0;
    }
    if (warp == 1) tmem_alloc(smem_u32(&s.tmem), TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // Only now may the next kernel start: one that took this SM's TMEM and then
    // waited for this kernel would never see it end.
    pdl_trigger();
    pdl_wait();
    if (warp == 0)
        expert_starts(c.offsets, c.E, c.R, BM, lane, s.start, s.tiles,
                      blockIdx.x == 0 ? c.status : nullptr);
    __syncthreads();

    const uint32_t tmem = s.tmem;
    constexpr int tile_cols = GATED ? BN / 2 : BN;
    const int nt = (c.epi.cols + tile_cols - 1) / tile_cols;
    const int64_t total = MODE == WGRAD
                              ? static_cast<int64_t>(c.E) * ((c.N + BM - 1) / BM) * nt
                              : static_cast<int64_t>(s.tiles[c.E]) * nt;
    constexpr uint32_t idesc = mma_desc(BM, BN, MODE == WGRAD, MODE != FWD);

    if (warp == 0) {
        if (lane == 0) {
            uint32_t n = 0;   // slices loaded so far
            for (int64_t t = blockIdx.x; t < total && !*gave_up; t += gridDim.x) {
                const Tile w = tile_at<MODE>(c, s.start, s.tiles, t, nt, tile_cols);
                for (int k = 0; k < w.depth; k += BK, ++n) {
                    const int i = n % STAGES;
                    if (!mbar_wait(smem_u32(&s.empty[i]), ((n / STAGES) & 1) ^ 1, gave_up)) break;
                    const uint32_t bar = smem_u32(&s.full[i]);
                    const uint32_t a = smem_u32(ring + i * STAGE_BYTES), b = a + A_BYTES;
                    mbar_expect(bar, STAGE_BYTES);
                    if (MODE == WGRAD) {
                        for (int j = 0; j < BM / 64; ++j)
                            tma_load(a + j * BOX_BYTES, &map_a, bar, w.m0 + 64 * j, w.row0 + k);
                        for (int j = 0; j < BN / 64; ++j)
                            tma_load(b + j * BOX_BYTES, &map_b, bar, w.c0 + 64 * j, w.row0 + k);
                    } else {
                        tma_load(a, &map_a, bar, k, w.m0);
                        if (MODE == FWD) {
                            tma_load(b, &map_b, bar, k, w.c0, w.e);
                            tma_load(b + B_BYTES / 2, &map_b, bar, k,
                                     GATED ? c.epi.cols + w.c0 : w.c0 + BN / 2, w.e);
                        } else {
                            for (int j = 0; j < BN / 64; ++j)
                                tma_load(b + j * BOX_BYTES, &map_b, bar, w.c0 + 64 * j, k, w.e);
                        }
                    }
                }
            }
            if (*gave_up)   // the copies still in flight end before the CTA does
                for (uint32_t q = n > STAGES ? n - STAGES : 0; q < n; ++q)
                    mbar_drain(smem_u32(&s.full[q % STAGES]), (q / STAGES) & 1);
        }
    } else if (warp == 1) {
        uint32_t n = 0, it = 0;   // slices and accumulators used so far
        bool ok = true;
        for (int64_t t = blockIdx.x; t < total && ok; t += gridDim.x) {
            const Tile w = tile_at<MODE>(c, s.start, s.tiles, t, nt, tile_cols);
            if (w.depth == 0) continue;
            const int acc = it & 1;
            ok = __all_sync(FULL_MASK, mbar_wait(smem_u32(&s.acc_empty[acc]), ((it >> 1) & 1) ^ 1, gave_up));
            if (!ok) break;
            tc_fence_after();
            const uint32_t d = tmem + acc * BN;
            for (int k = 0; k < w.depth; k += BK, ++n) {
                const int i = n % STAGES;
                ok = __all_sync(FULL_MASK, mbar_wait(smem_u32(&s.full[i]), (n / STAGES) & 1, gave_up));
                if (!ok) break;
                uint8_t *tile = ring + i * STAGE_BYTES;
                int steps = BK / 16;
                if (MODE == WGRAD && k + BK > w.depth) {
                    const int rows = w.depth - k;
                    steps = (rows + 15) / 16;
                    // Rows [rows, 16 steps) of the six boxes: 128 bytes each, whatever the swizzle.
                    for (int v = lane; v < (16 * steps - rows) * (STAGE_BYTES / BOX_BYTES) * 8; v += 32) {
                        const int row = rows + (v >> 3) % (16 * steps - rows);
                        const int box = (v >> 3) / (16 * steps - rows);
                        *reinterpret_cast<uint4 *>(tile + box * BOX_BYTES + row * 128 + (v & 7) * 16) =
                            make_uint4(0, 0, 0, 0);
                    }
                    fence_async_smem();
                    __syncwarp();
                }
                tc_fence_after();
                if (lane == 0) {
                    const uint32_t a = smem_u32(tile), b = a + A_BYTES;
                    for (int q = 0; q < steps; ++q)
                        tc_mma(d, tile_desc(a + q * (MODE == WGRAD ? 2048 : 32), BOX_BYTES),
                               tile_desc(b + q * (MODE == FWD ? 32 : 2048), BOX_BYTES), idesc,
                               (k | q) != 0);
                    tc_commit(smem_u32(&s.empty[i]));
                }
                __syncwarp();
            }
            if (ok && lane == 0) tc_commit(smem_u32(&s.acc_full[acc]));
            __syncwarp();
            ++it;
        }
        if (!ok && lane == 0) {
            tc_commit(smem_u32(&s.drained));
            mbar_drain(smem_u32(&s.drained), 0);
            or_status(c.status, MP_STATUS_STALLED);
        }
    } else {
        const int quad = warp & 3;            // the TMEM lanes this warp can read
        const int half = (warp - 2) >> 2;     // and its half of the columns
        WarpWriter out = {ring + STAGES * STAGE_BYTES + (warp - 2) * STAGING, stores, lane, 0};
        uint32_t it = 0;
        for (int64_t t = blockIdx.x; t < total; t += gridDim.x) {
            const Tile w = tile_at<MODE>(c, s.start, s.tiles, t, nt, tile_cols);
            if (MODE == WGRAD && w.depth == 0 && c.epi.add) continue;   // nothing to add
            out.rows = min(w.m1 - (w.m0 + quad * 32), 32);
            const bool valid = lane < out.rows;
            const int row = min(w.m0 + quad * 32 + lane, w.m1 - 1);   // lanes past the end read the last
            const int acc = it & 1;
            const int j0 = half * (tile_cols / 2), j1 = j0 + tile_cols / 2;
            if (MODE != WGRAD && valid && w.c0 + j0 < c.epi.cols)
                epi_prefetch<MODE>(c.epi, row, w.c0 + j0, min(w.c0 + j1, c.epi.cols));
            if (w.depth != 0) {
                if (!__all_sync(FULL_MASK, mbar_wait(smem_u32(&s.acc_full[acc]), (it >> 1) & 1, gave_up)))
                    break;
                tc_fence_after();
            }
            const uint32_t d = tmem + acc * BN + (static_cast<uint32_t>(quad * 32) << 16);
            for (int j = j0; j < j1; j += EPI_COLS) {
                const int col = w.c0 + j;
                if (col >= c.epi.cols) break;
                float z[EPI_COLS], u[EPI_COLS];
                if (w.depth != 0) {
                    tmem_load32(d + j, z);
                    if (GATED) tmem_load32(d + BN / 2 + j, u);
                    tmem_load_wait();
                } else {
#pragma unroll
                    for (int i = 0; i < EPI_COLS; ++i) z[i] = 0.0f;
                }
                if (out.rows > 0) {
                    const int n = min(EPI_COLS, c.epi.cols - col);
                    if (MODE == FWD) epi_fwd<GATED>(c.epi, out, w.e, row, col, n, valid, z, u);
                    if (MODE == DGRAD) epi_dgrad(c.epi, out, row, col, n, valid, z);
                    if (MODE == WGRAD)
                        epi_wgrad(c.epi, out, static_cast<int64_t>(w.e) * c.N + row, col, n, valid, z);
                }
                __syncwarp();
            }
            if (w.depth != 0) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&s.acc_empty[acc]));
                ++it;
            }
        }
        if (lane == 0) tma_store_done();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_free(tmem, TMEM_COLS);
    }
}

// The map of a result of `rows` rows of parts * cols, where TMA can address it:
// every part starts on a 16-byte boundary.
bool store_map(StoreMaps &m, int which, const void *base, int64_t parts, int64_t cols, int64_t rows)
{
    const int64_t pitch = parts * cols;
    const uint64_t dims[2] = {static_cast<uint64_t>(pitch), static_cast<uint64_t>(rows)};
    const uint32_t box[2] = {EPI_COLS, 32};
    m.use[which] = base != nullptr && cols % 8 == 0 && aligned16(base) && rows <= INT32_MAX;
    return !m.use[which] || make_map(&m.map[which], base, 2, dims, box);
}

template <int MODE, bool GATED> mp_status_t launch_tc(const ExpertCall &c, const CUtensorMap &a,
                                                      const CUtensorMap &b, const StoreMaps &m)
{
    static std::atomic<uint64_t> allowed{0};
    if (!allow_smem(k_expert_tc<MODE, GATED>, allowed, TC_SMEM)) return MP_ERR_CUDA;
    const int64_t nt = (c.epi.cols + (GATED ? BN / 2 : BN) - 1) / (GATED ? BN / 2 : BN);
    const int64_t mt = MODE == WGRAD ? static_cast<int64_t>(c.E) * ((c.N + BM - 1) / BM)
                                     : c.R / BM + (c.R < c.E ? c.R : c.E);
    const int64_t tiles = nt * mt, sms = sm_count();
    (void)launch_pdl(k_expert_tc<MODE, GATED>, static_cast<unsigned>(tiles < sms ? tiles : sms),
                     TC_THREADS, TC_SMEM, c.stream, a, b, m, c);
    return check_launch();
}

}  // namespace

template <int MODE> bool expert_tc_takes(const ExpertCall &c)
{
    return c.R > 0 && c.K % 8 == 0 && (MODE == FWD || c.N % 8 == 0) && aligned16(c.a) && aligned16(c.b);
}

template <int MODE> mp_status_t expert_tc(const ExpertCall &c)
{
    CUtensorMap a, b;
    const uint64_t R = c.R, N = c.N, K = c.K, E = c.E;
    const uint64_t da[2] = {MODE == FWD ? K : N, R};
    const uint32_t box_a[2] = {64, MODE == WGRAD ? 64u : static_cast<uint32_t>(BM)};
    const uint64_t db[3] = {K, MODE == WGRAD ? R : N, E};
    const uint32_t box_b[3] = {64, MODE == FWD ? BN / 2u : 64u, 1};
    if (!make_map(&a, c.a, 2, da, box_a) || !make_map(&b, c.b, MODE == WGRAD ? 2 : 3, db, box_b)) {
        set_last_cuda_error(cudaErrorInvalidValue);
        return MP_ERR_CUDA;
    }
    StoreMaps m = {};
    const int64_t cols = c.epi.cols, parts = act_gated(c.epi.act) ? 2 : 1;
    const bool ok =
        store_map(m, TO_OUT, c.epi.out, MODE == DGRAD ? parts : 1, cols,
                  MODE == WGRAD ? static_cast<int64_t>(c.E) * c.N : c.R) &&
        (MODE != FWD || c.epi.save != MP_SAVE_BF16 || store_map(m, TO_SECOND, c.epi.z, parts, cols, c.R)) &&
        (MODE != DGRAD || store_map(m, TO_SECOND, c.epi.h, 1, cols, c.R));
    if (!ok) {
        set_last_cuda_error(cudaErrorInvalidValue);
        return MP_ERR_CUDA;
    }
    if (MODE == FWD && act_gated(c.epi.act)) return launch_tc<MODE, MODE == FWD>(c, a, b, m);
    return launch_tc<MODE, false>(c, a, b, m);
}

template bool expert_tc_takes<FWD>(const ExpertCall &);
template bool expert_tc_takes<DGRAD>(const ExpertCall &);
template bool expert_tc_takes<WGRAD>(const ExpertCall &);
template mp_status_t expert_tc<FWD>(const ExpertCall &);
template mp_status_t expert_tc<DGRAD>(const ExpertCall &);
template mp_status_t expert_tc<WGRAD>(const ExpertCall &);

}  // namespace mp
