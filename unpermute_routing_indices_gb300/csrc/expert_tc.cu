// The experts' products on the tensor cores.
//
// One persistent kernel for the three products, a CTA per SM.  A tile is 128
// rows by up to 256 columns (half of them the gate's when gated) of one expert,
// or 256 rows and columns for a pair of CTAs, which read half of B each:
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
// Operands that TMA cannot address (rows that are no multiple of 16 bytes, or begin
// off them) are read by four more warps, word by word, into the same layout: 24,576
// rows by 64 experts of 2,046 x 2,045 in 1,033 us (200 TFLOP/s; an element a lane with
// 64-bit addresses 3,500), of 2,048 x 2,048 by TMA in 160.
// Where the tiles are few, they are narrower (choose_cut), and the contraction of
// each may be split over a cluster of up to 8 CTAs, whose parts are added in rank order
// through distributed shared memory, so a result does not depend on timing.
// What bounds it: for experts of many rows the tensor cores (131,072 x 4,096 by 128
// experts of 2,048 columns, swiglu: in short runs on equal loads 1,211 us, 1.82 PFLOP/s,
// 0.92 of cuBLAS's measured 8,192^3; on unequal loads and under the power limit 1,490 to
// 1,560 us, 1.41 to 1.48); for few rows the bytes of weights and results and the epilogue.
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

constexpr int BM = 128, BN = 256, BK = 64;   // one CTA's rows, columns, depth of a slice
constexpr int A_BYTES = BM * BK * 2;
constexpr int BOX_BYTES = 64 * 64 * 2;       // a box of 64 rows
constexpr int TMEM_COLS = 2 * BN;
// CG CTAs share a tile of CG * 128 rows and 256 columns; each holds 256 / CG rows
// of B.
template <int CG> struct Ring {
    static constexpr int STAGES = CG == 1 ? 4 : 6;
    static constexpr int B_BYTES = BN / CG * BK * 2;
    static constexpr int STAGE = A_BYTES + B_BYTES;
};
constexpr int RING_BYTES = Ring<1>::STAGES * Ring<1>::STAGE;
static_assert(RING_BYTES == Ring<2>::STAGES * Ring<2>::STAGE, "one layout");
constexpr int MOST_STAGES = 6;
constexpr int EPI_WARPS = 8;   // two for each quarter of the accumulator's lanes
constexpr int SUM_WARPS = 4;   // WGRAD: column sums for the bias gradient
constexpr int LOAD_WARPS = 4;  // operands that TMA cannot address
__host__ __device__ constexpr int tc_threads(int mode, bool raw)
{
    return 64 + 32 * (EPI_WARPS + (raw ? LOAD_WARPS : mode == WGRAD ? SUM_WARPS : 0));
}
constexpr int STAGING = 32 * EPI_COLS * 2;   // bytes of one warp's tile on its way out

struct TcShared {
    uint64_t full[MOST_STAGES], peer_full[MOST_STAGES], empty[MOST_STAGES], acc_full[2], acc_empty[2], drained;
    uint32_t tmem;
    int gave_up;
    uint32_t loaded;   // slices that this CTA has begun to load: what the waits for a contraction go by
    float sums[SUM_WARPS][BM], sum[BM];
    int start[MP_MAX_EXPERTS + 1], tiles[MP_MAX_EXPERTS + 1];
};
constexpr size_t TC_SMEM = 1024 + RING_BYTES + EPI_WARPS * STAGING + sizeof(TcShared);
static_assert(TC_SMEM <= 232448, "shared memory of one SM");

struct Tile {
    int e, m0, m1, c0, row0, depth;   // rows from m0 (this CTA's) up to m1 of the result (of g's columns in WGRAD)
    int k0, k1;                       // this CTA's part of the contraction, whole slices but its end
};

template <int MODE, int CG>
__device__ __forceinline__ Tile tile_at(const ExpertCall &c, const int *start, const int *tiles,
                                        int t, int nt, int tile_cols, int rank, int part, int parts)
{
    constexpr int TM = CG * BM;
    Tile r;
    int at, mt;   // the tile's place among its expert's, which are mt high
    if (MODE == WGRAD) {
        mt = (c.N + TM - 1) / TM;
        r.e = t / (mt * nt);
        at = t - r.e * (mt * nt);
    } else {
        r.e = expert_of_tile(tiles, c.E, t / nt);
        mt = tiles[r.e + 1] - tiles[r.e];
        at = t - tiles[r.e] * nt;
    }
    const int column = at / mt, m0 = (at - column * mt) * TM + rank * BM;
    r.c0 = column * tile_cols;
    if (MODE == WGRAD) {
        r.m0 = m0;
        r.m1 = c.N;
        r.row0 = start[r.e];
        r.depth = start[r.e + 1] - r.row0;
    } else {
        r.m0 = start[r.e] + m0;
        r.m1 = start[r.e + 1];
        r.row0 = 0;
        r.depth = MODE == FWD ? c.K : c.N;
    }
    r.k0 = 0;
    r.k1 = r.depth;
    if (parts > 1) {
        const int slices = (r.depth + BK - 1) / BK;   // at most 2^25, and parts at most 8
        r.k0 = slices * part / parts * BK;
        r.k1 = min(slices * (part + 1) / parts * BK, r.depth);
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
            *piece(lane, q) = pack8(f + 8 * q);
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
        if (n % 8 == 0 && maps.use[which]) {
            if ((lane & 3) * 8 < n)
#pragma unroll 4
                for (int r = lane >> 2; r < rows; r += 8)
                    *reinterpret_cast<uint4 *>(to + r * pitch + (lane & 3) * 8) = *piece(r, lane & 3);
        } else if (lane < n) {
#pragma unroll 8
            for (int r = 0; r < rows; ++r) to[r * pitch + lane] = *element(r, lane);
        }
    }
    __device__ __forceinline__ uint4 *piece(int r, int q)
    {
        return reinterpret_cast<uint4 *>(tile + r * 64 + ((q ^ ((r >> 1) & 3)) * 16));
    }
    __device__ __forceinline__ uint16_t *element(int r, int col)
    {
        return reinterpret_cast<uint16_t *>(piece(r, col >> 3)) + (col & 7);
    }
    // Rows whose 32-byte sectors a lane cannot read whole are read as they are written,
    // and turned: 20,000 rows by 64 experts of 1,016 x 1,024 with a residual 87 -> 65 us,
    // 2,999 rows by 40 experts of 1,009 x 1,000 106 -> 41.
    // WRITTEN: what is read may be what the kernel writes, each element after it is read.
    template <bool WRITTEN>
    __device__ __forceinline__ void get(const mp_bf16_t *base, int64_t pitch, int64_t row, int64_t c, int n,
                                        float (&f)[EPI_COLS])
    {
        const unsigned low = low_bits(base) | ((static_cast<unsigned>(pitch | c) & 15u) * 2);
        if (n == EPI_COLS && low == 0) {
            load32<WRITTEN>(base + row * pitch + c, f);
            return;
        }
        if (lane == 0) tma_store_read();   // the tile before this one has left
        __syncwarp();
        const mp_bf16_t *from = base + __shfl_sync(FULL_MASK, row, 0) * pitch + c;
        if (n % 8 == 0 && (low & 15u) == 0) {
            uint4 v[4] = {};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = (lane >> 2) + 8 * i;
                if (r < rows && (lane & 3) * 8 < n)
                    v[i] = ld_of<WRITTEN>(reinterpret_cast<const uint4 *>(from + r * pitch) + (lane & 3));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) *piece((lane >> 2) + 8 * i, lane & 3) = v[i];
        } else {
            uint16_t v[32] = {};
#pragma unroll
            for (int r = 0; r < 32; ++r)
                if (r < rows && lane < n) v[r] = ld_of<WRITTEN>(from + r * pitch + lane);
#pragma unroll
            for (int r = 0; r < 32; ++r) *element(r, lane) = v[r];
        }
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float t[8];
            unpack(*piece(lane, q), t);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[8 * q + i] = t[i];
        }
        __syncwarp();
    }
    // The same values for all the rows.
    __device__ __forceinline__ void get_shared(const mp_bf16_t *p, int n, float (&f)[EPI_COLS])
    {
        if (n == EPI_COLS && (low_bits(p) & 15u) == 0) {   // from L1 but for the first of four warps
            const uint4 *q = reinterpret_cast<const uint4 *>(p);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float t[8];
                unpack(__ldg(q + j), t);
#pragma unroll
                for (int i = 0; i < 8; ++i) f[8 * j + i] = t[i];
            }
            return;
        }
        float t[1] = {0.0f};
        if (lane < n) unpack(__ldg(p + lane), t);
#pragma unroll
        for (int i = 0; i < EPI_COLS; ++i) f[i] = __shfl_sync(FULL_MASK, t[0], i);
    }
};

// A slice of `rows` rows, contraction across them: zeroes the rows up to the next
// 16 in every box (128 bytes each, whatever the swizzle), for the products to read,
// and returns how many steps of 16 there are.
template <int CG> __device__ __forceinline__ int zero_ragged(uint8_t *tile, int rows, int lane)
{
    const int steps = (rows + 15) / 16;
    uint8_t *piece = tile + (lane >> 3) * BOX_BYTES + (lane & 7) * 16;   // four boxes at a time
    for (int row = rows; row < 16 * steps; ++row)
#pragma unroll
        for (int box = 0; box < Ring<CG>::STAGE / BOX_BYTES; box += 4)
            if (box + (lane >> 3) < Ring<CG>::STAGE / BOX_BYTES)
                *reinterpret_cast<uint4 *>(piece + box * BOX_BYTES + row * 128) = make_uint4(0, 0, 0, 0);
    fence_async_smem();
    __syncwarp();
    return steps;
}

// A load that its predicate may leave out, without a branch.
__device__ __forceinline__ uint32_t ld_word_if(const uint32_t *p, bool there)
{
    uint32_t v;
    asm volatile("{\n\t.reg .pred there;\n\tsetp.ne.u32 there, %2, 0;\n\tmov.u32 %0, 0;\n\t"
                 "@there ld.global.nc.u32 %0, [%1];\n\t}"
                 : "=r"(v)
                 : "l"(p), "r"(static_cast<uint32_t>(there)));
    return v;
}

// 8 neighbouring elements of which the first n exist, zeros in place of the others,
// by loads of the aligned words that hold them (no word without one is read).
struct Piece {
    int shift, words;   // 16: the first element is the upper half of the first word
    uint32_t mask[4];
    __device__ __forceinline__ Piece(const mp_bf16_t *p, int n)
    {
        const int odd = (reinterpret_cast<uintptr_t>(p) >> 1) & 1;
        shift = 16 * odd;
        n = min(max(n, 0), 8);
        words = n == 0 ? 0 : (odd + n + 1) >> 1;
#pragma unroll
        for (int i = 0; i < 4; ++i) mask[i] = n >= 2 * i + 2 ? 0xffffffffu : n == 2 * i + 1 ? 0xffffu : 0u;
    }
    __device__ __forceinline__ void load(uint32_t (&v)[5], const uint32_t *q, bool there) const
    {
#pragma unroll
        for (int i = 0; i < 5; ++i) v[i] = ld_word_if(q + i, there && i < words);
    }
    __device__ __forceinline__ uint4 value(const uint32_t (&v)[5]) const
    {
        return make_uint4(__funnelshift_r(v[0], v[1], shift) & mask[0], __funnelshift_r(v[1], v[2], shift) & mask[1],
                          __funnelshift_r(v[2], v[3], shift) & mask[2], __funnelshift_r(v[3], v[4], shift) & mask[3]);
    }
};

__device__ __forceinline__ const uint32_t *word_of(const mp_bf16_t *p)
{
    return reinterpret_cast<const uint32_t *>(reinterpret_cast<uintptr_t>(p) & ~static_cast<uintptr_t>(3));
}

// Operands by loads, as TMA would place them: row r of 64 columns at r * 128 bytes,
// its 16-byte pieces swizzled, zeros for what is not there.  A thread has a piece of
// every 16th row, so that all of its pieces begin in the same half of a word, and
// eight in flight.  `from`: this thread's piece of row 0; n: elements from there on.
constexpr int RAW_STEP = 32 * LOAD_WARPS / 8;
static_assert(RAW_STEP == 16, "four pieces of a box of 64 rows a thread");

// `total` rows, of which `rows` exist.
__device__ __forceinline__ void load_rows(uint8_t *to, const mp_bf16_t *from, int64_t pitch, int rows, int total,
                                          int n, int t, int q)
{
    from += t * pitch;
    const Piece piece(from, n);
    const uint32_t *word = word_of(from);
    for (int r0 = t; r0 < total; r0 += 8 * RAW_STEP) {
        uint32_t v[8][5];
#pragma unroll
        for (int i = 0; i < 8; ++i, word += RAW_STEP / 2 * pitch) piece.load(v[i], word, r0 + RAW_STEP * i < rows);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = r0 + RAW_STEP * i;
            if (r < total) *reinterpret_cast<uint4 *>(to + r * 128 + ((q ^ (r & 7)) * 16)) = piece.value(v[i]);
        }
    }
}

// `boxes` of 64 rows of 64 columns side by side, of whose rows `rows` exist.
__device__ __forceinline__ void load_boxes(uint8_t *to, const mp_bf16_t *from, int64_t pitch, int rows, int boxes,
                                           int n, int t, int q)
{
    from += t * pitch;
    const uint32_t *word = word_of(from);
    for (int box = 0; box < boxes; box += 2, word += 64) {
        const Piece left(from, n - 64 * box), right(from, box + 1 < boxes ? n - 64 * box - 64 : 0);
        uint32_t v[8][5];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            (i < 4 ? left : right).load(v[i], word + (i & 3) * (RAW_STEP / 2) * pitch + (i >> 2) * 32,
                                        t + RAW_STEP * (i & 3) < rows);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = t + RAW_STEP * (i & 3);
            if (i < 4 || box + 1 < boxes)
                *reinterpret_cast<uint4 *>(to + (box + (i >> 2)) * BOX_BYTES + r * 128 + ((q ^ (r & 7)) * 16)) =
                    (i < 4 ? left : right).value(v[i]);
        }
    }
}

// The slice at depth k, by thread `tid` of the load warps.
template <int MODE, bool GATED>
__device__ __forceinline__ void load_slice(const ExpertCall &c, const Tile &w, uint8_t *a, int k, int wide, int tid)
{
    const int q = tid & 7, t = tid >> 3, col = k + 8 * q;
    uint8_t *b = a + A_BYTES;
    if (MODE == WGRAD) {
        const int64_t row = static_cast<int64_t>(w.row0) + k;
        const int rows = w.depth - k, am = w.m0 + 8 * q, bn = w.c0 + 8 * q;
        load_boxes(a, c.a + row * c.N + am, c.N, rows, BM / 64, c.N - am, t, q);
        load_boxes(b, c.b + row * c.K + bn, c.K, rows, wide / 64, c.K - bn, t, q);
        return;
    }
    const int pitch = MODE == FWD ? c.K : c.N;   // of A
    load_rows(a, c.a + static_cast<int64_t>(w.m0) * pitch + col, pitch, w.m1 - w.m0, BM, pitch - col, t, q);
    const mp_bf16_t *weights = c.b + static_cast<int64_t>(w.e) * c.N * c.K;
    if (MODE == FWD) {
        const mp_bf16_t *from = weights + static_cast<int64_t>(w.c0) * c.K + col;
        const int high = GATED ? wide / 2 : wide;
        load_rows(b, from, c.K, c.epi.cols - w.c0, high, c.K - col, t, q);
        if (GATED)
            load_rows(b + high * 128, from + static_cast<int64_t>(c.epi.cols) * c.K, c.K, c.epi.cols - w.c0, high,
                      c.K - col, t, q);
    } else {
        const int bn = w.c0 + 8 * q;
        load_boxes(b, weights + static_cast<int64_t>(k) * c.K + bn, c.K, c.N - k, wide / 64, c.K - bn, t, q);
    }
}

// The sum warps alone.
__device__ __forceinline__ void sums_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * SUM_WARPS) : "memory"); }

// The bias gradient of a tile's 128 columns of g: column sums over the expert's
// rows, by warps that wait for nothing else, beside the product.  A thread has 8
// columns of every eighth row, eight rows in flight; the sums of a warp, then of the
// warps, are added in order.  256 experts of 128 rows, 1,024 x 2,048: a kernel of
// its own after this one took 28 us more, the epilogue warps doing it 24.
__device__ __forceinline__ float column_sum(const ExpertCall &c, const Tile &w, float (&sums)[SUM_WARPS][BM], int tid)
{
    constexpr int ROWS = 2 * SUM_WARPS, DEEP = 8;
    const int col = w.m0 + (tid & 15) * 8, warp = tid >> 5;
    float s[8] = {};
    if (col < c.N) {
        const uint4 *p = reinterpret_cast<const uint4 *>(c.a + static_cast<int64_t>(w.row0) * c.N + col);
        const int64_t pitch = c.N / 8;
        for (int r = w.k0 + (tid >> 4); r < w.k1; r += DEEP * ROWS) {
            uint4 v[DEEP];
#pragma unroll
            for (int q = 0; q < DEEP; ++q)
                v[q] = r + ROWS * q < w.k1 ? ld_stream(p + (r + ROWS * q) * pitch) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int q = 0; q < DEEP; ++q) {
                float f[8];
                unpack(v[q], f);
#pragma unroll
                for (int i = 0; i < 8; ++i) s[i] += f[i];
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] += __shfl_xor_sync(FULL_MASK, s[i], 16);
    sums_sync();   // the sums of the tile before have been read
    if ((tid & 31) < 16) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sums[warp][(tid & 15) * 8 + i] = s[i];
    }
    sums_sync();
    float t = sums[0][tid];
    for (int q = 1; q < SUM_WARPS; ++q) t += sums[q][tid];
    return t;
}

__device__ __forceinline__ void put_bias_grad(const ExpertCall &c, const Tile &w, int tid, float t)
{
    if (w.m0 + tid >= c.N) return;
    const int64_t at = static_cast<int64_t>(w.e) * c.N + w.m0 + tid;
    if (c.epi.g_bias_f32 != nullptr) {
        c.epi.g_bias_f32[at] = c.epi.add ? c.epi.g_bias_f32[at] + t : t;
    } else {
        const float f[1] = {t};
        c.epi.g_bias[at] = pack(f);
    }
}
static_assert(32 * SUM_WARPS == BM, "a column a thread");

// The epilogue of 32 columns, from j, of the 32 rows of a tile's quarter.
template <int MODE, bool GATED>
__device__ __forceinline__ void finish(const ExpertCall &c, WarpWriter &out, const Tile &w, int quad, int j,
                                       float (&z)[EPI_COLS], float (&u)[EPI_COLS])
{
    out.rows = min(w.m1 - (w.m0 + quad * 32), 32);
    if (out.rows <= 0) return;
    const bool valid = out.lane < out.rows;
    const int row = min(w.m0 + quad * 32 + out.lane, w.m1 - 1);   // lanes past the end read the last
    const int col = w.c0 + j, n = min(EPI_COLS, c.epi.cols - col);
    if (MODE == FWD) epi_fwd<GATED>(c.epi, out, w.e, row, col, n, valid, z, u);
    if (MODE == DGRAD) epi_dgrad(c.epi, out, row, col, n, valid, z);
    if (MODE == WGRAD) epi_wgrad(c.epi, out, static_cast<int64_t>(w.e) * c.N + row, col, n, valid, z);
}

// Floats of a row of a CTA's part of a split tile; 8 rows on different banks.
constexpr int JOIN_PITCH = BN + 4;
constexpr int JOIN_BYTES = BM * JOIN_PITCH * 4, TURN_BYTES = 32 * 33 * 4;
static_assert(JOIN_BYTES + EPI_WARPS * TURN_BYTES <= RING_BYTES, "a part, and a turn for each warp, fit the ring");

__device__ __forceinline__ float peer_float(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
// Sums 32 rows of 32 floats over the ranks, in rank order: a lane reads a column, so
// that every load is a line of the peer's memory (a row a lane, 16 bytes each, took
// 25 us more for a cluster of 8), and gets its row through `turn`.
__device__ __forceinline__ void join32(uint32_t addr, int split, float *turn, int lane, float (&z)[EPI_COLS])
{
#pragma unroll
    for (int i = 0; i < 32; ++i) z[i] = 0.0f;
    for (int r = 0; r < split; ++r) {
        const uint32_t from = at_rank(addr, r) + lane * 4;
        float v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = peer_float(from + i * JOIN_PITCH * 4);
#pragma unroll
        for (int i = 0; i < 32; ++i) z[i] += v[i];
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 32; ++i) turn[i * 33 + lane] = z[i];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 32; ++i) z[i] = turn[lane * 33 + i];
}

// ANY: tiles of `width` columns; otherwise of BN, which the weight gradients of many
// experts would feel (64 experts of 384 rows, 2,048 x 2,048: 191 us, as a variable 195).
// RAW: operands of any alignment and width, by load_slice.
template <int MODE, bool GATED, int CG, bool ANY, bool RAW = false>
__global__ void __launch_bounds__(tc_threads(MODE, RAW), 1)
    k_expert_tc(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                const __grid_constant__ StoreMaps stores, const ExpertCall c, int split, int width)
{
    typedef Ring<CG> L;
    constexpr int STAGES = L::STAGES;
    extern __shared__ uint8_t raw[];
    uint8_t *ring = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    TcShared &s = *reinterpret_cast<TcShared *>(ring + RING_BYTES + EPI_WARPS * STAGING);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = CG == 2 ? static_cast<int>(cluster_rank()) : 0;
    const int part = CG == 1 && split > 1 ? static_cast<int>(cluster_rank()) : 0;
    volatile int *gave_up = &s.gave_up;
    volatile uint32_t *loaded = &s.loaded;

    if (threadIdx.x == 0) {
        if (!RAW) {
            tma_prefetch(&map_a);
            tma_prefetch(&map_b);
        }
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(smem_u32(&s.full[i]), RAW ? LOAD_WARPS : 1);
            mbar_init(smem_u32(&s.peer_full[i]), 1);
            mbar_init(smem_u32(&s.empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&s.acc_full[i]), 1);
            mbar_init(smem_u32(&s.acc_empty[i]), CG * EPI_WARPS);
        }
        mbar_init(smem_u32(&s.drained), 1);
        mbar_init_fence();
        s.gave_up = 0;
        s.loaded = 0;
    }
    __syncwarp();
    if (warp == 1) tmem_alloc<CG>(smem_u32(&s.tmem), TMEM_COLS);
    tc_fence_before();
    if (CG == 2)
        cluster_sync();   // the other CTA's barriers exist
    else
        __syncthreads();
    tc_fence_after();
    // Only now may the next kernel start: one that took this SM's TMEM and then
    // waited for this kernel would never see it end.
    pdl_trigger();
    pdl_wait();
    if (warp == 0)
        expert_starts(c.offsets, c.E, c.R, CG * BM, lane, s.start, s.tiles,
                      blockIdx.x == 0 ? c.status : nullptr);
    __syncthreads();

    const uint32_t tmem = s.tmem;
    const int wide = ANY ? width : BN;   // columns of B's slice and of the accumulator
    const int tile_cols = GATED ? wide / 2 : wide;
    const int nt = (c.epi.cols + tile_cols - 1) / tile_cols;
    const int total = (MODE == WGRAD ? c.E * ((c.N + CG * BM - 1) / (CG * BM)) : s.tiles[c.E]) * nt;
    const int first = blockIdx.x / (CG * split), step = gridDim.x / (CG * split);
    const uint32_t idesc = mma_desc(CG * BM, wide, MODE == WGRAD, MODE != FWD);
    const uint32_t slice_bytes = A_BYTES + wide / CG * BK * 2;

    if (warp == 0) {
        if (!RAW && lane == 0) {
            uint32_t n = 0;   // slices loaded so far
            for (int t = first; t < total && !*gave_up; t += step) {
                const Tile w = tile_at<MODE, CG>(c, s.start, s.tiles, t, nt, tile_cols, rank, part, split);
                const int off = rank * (wide / 2);   // in B's rows or columns
                for (int k = w.k0; k < w.k1; k += BK, ++n) {
                    const int i = n % STAGES;
                    if (!mbar_wait(smem_u32(&s.empty[i]), ((n / STAGES) & 1) ^ 1, gave_up)) break;
                    *loaded = n + 1;
                    uint32_t bar = smem_u32(&s.full[i]);
                    const uint32_t a = smem_u32(ring + i * L::STAGE), b = a + A_BYTES;
                    // In a pair both CTAs' copies arrive at CTA 0's barrier, but those
                    // of a ragged slice, which CTA 1 has to see itself.
                    if (CG == 1 || (MODE == WGRAD && k + BK > w.depth))
                        mbar_expect(bar, slice_bytes);
                    else if (rank == 0)
                        mbar_expect(bar, 2 * slice_bytes);
                    else
                        bar = at_rank(bar, 0);
                    if (MODE == WGRAD) {
                        for (int j = 0; j < BM / 64; ++j)
                            tma_load<CG>(a + j * BOX_BYTES, &map_a, bar, w.m0 + 64 * j, w.row0 + k);
                        for (int j = 0; j < wide / CG / 64; ++j)
                            tma_load<CG>(b + j * BOX_BYTES, &map_b, bar, w.c0 + off + 64 * j, w.row0 + k);
                    } else {
                        // A part without rows reads zeros from past the end of x: the
                        // products are made all the same, but on less power and no bytes.
                        tma_load<CG>(a, &map_a, bar, k, w.m0 < w.m1 ? w.m0 : c.R);
                        if (MODE == FWD) {
                            // Half the rows of w at a time: the gate's and the others', or neighbours.
                            for (int j = rank; j < rank + 2 / CG; ++j)
                                tma_load<CG>(b + (j - rank) * (wide / 2) * BK * 2, &map_b, bar, k,
                                             w.c0 + j * (GATED ? c.epi.cols : wide / 2), w.e);
                        } else {
                            for (int j = 0; j < wide / CG / 64; ++j)
                                tma_load<CG>(b + j * BOX_BYTES, &map_b, bar, w.c0 + off + 64 * j, k, w.e);
                        }
                    }
                }
            }
            if (*gave_up) {   // the copies still in flight end before the CTA does
                if (rank == 0) {
                    for (uint32_t q = n > STAGES ? n - STAGES : 0; q < n; ++q)
                        mbar_drain(smem_u32(&s.full[q % STAGES]), (q / STAGES) & 1);
                } else {   // theirs are the other CTA's barriers: wait by the clock
                    const uint64_t t0 = now_ns();
                    while (now_ns() - t0 < 100000000ull) __nanosleep(1000);
                }
            }
        }
    } else if (warp == 1 && rank == 0) {
        uint32_t n = 0, it = 0;   // slices and accumulators used so far
        uint32_t ragged = 0;      // bit i: the phase of stage i's ragged slices
        bool ok = true;
        for (int t = first; t < total && ok; t += step) {
            const Tile w = tile_at<MODE, CG>(c, s.start, s.tiles, t, nt, tile_cols, rank, part, split);
            if (w.k0 >= w.k1) continue;
            const int acc = it & 1;
            ok = __all_sync(FULL_MASK, mbar_wait(smem_u32(&s.acc_empty[acc]), ((it >> 1) & 1) ^ 1, gave_up));
            if (!ok) break;
            tc_fence_after();
            const uint32_t d = tmem + acc * BN;
            for (int k = w.k0; k < w.k1; k += BK, ++n) {
                const int i = n % STAGES;
                ok = __all_sync(FULL_MASK, mbar_wait(smem_u32(&s.full[i]), (n / STAGES) & 1, gave_up));
                if (!ok) break;
                uint8_t *tile = ring + i * L::STAGE;
                int steps = BK / 16;
                if (MODE == WGRAD && k + BK > w.depth) {
                    steps = RAW ? (w.depth - k + 15) / 16 : zero_ragged<CG>(tile, w.depth - k, lane);
                    if (CG == 2) {
                        ok = __all_sync(FULL_MASK, mbar_wait(smem_u32(&s.peer_full[i]), (ragged >> i) & 1, gave_up));
                        if (!ok) break;
                        ragged ^= 1u << i;
                    }
                }
                tc_fence_after();
                if (lane == 0) {
                    const uint32_t a = smem_u32(tile), b = a + A_BYTES;
                    for (int q = 0; q < steps; ++q)
                        tc_mma<CG>(d, tile_desc(a + q * (MODE == WGRAD ? 2048 : 32), BOX_BYTES),
                                   tile_desc(b + q * (MODE == FWD ? 32 : 2048), BOX_BYTES), idesc,
                                   k != w.k0 || q != 0);
                    tc_commit<CG>(smem_u32(&s.empty[i]));
                }
                __syncwarp();
            }
            if (ok && lane == 0) tc_commit<CG>(smem_u32(&s.acc_full[acc]));
            __syncwarp();
            ++it;
        }
        if (!ok && lane == 0) {
            tc_commit<CG>(smem_u32(&s.drained));
            mbar_drain(smem_u32(&s.drained), 0);
            or_status(c.status, MP_STATUS_STALLED);
        }
    } else if (warp == 1 && MODE == WGRAD) {
        // CTA 1 of a pair: zeroes its part of the ragged slices, and says so.
        uint32_t n = 0, ragged = 0;
        bool ok = true;
        for (int t = first; t < total && ok; t += step) {
            const Tile w = tile_at<MODE, CG>(c, s.start, s.tiles, t, nt, tile_cols, rank, part, split);
            n += (w.depth + BK - 1) / BK;
            if (w.depth % BK == 0) continue;
            const int i = (n - 1) % STAGES;
            ok = __all_sync(FULL_MASK, mbar_wait(smem_u32(&s.full[i]), (ragged >> i) & 1, gave_up, loaded));
            if (!ok) break;
            ragged ^= 1u << i;
            zero_ragged<CG>(ring + i * L::STAGE, w.depth % BK, lane);
            if (lane == 0) mbar_arrive_cluster(at_rank(smem_u32(&s.peer_full[i]), 0));
            __syncwarp();
        }
        if (!ok && lane == 0) or_status(c.status, MP_STATUS_STALLED);
    } else if (RAW && warp >= 2 + EPI_WARPS) {
        const int tid = threadIdx.x - 64 - 32 * EPI_WARPS;
        uint32_t n = 0;
        bool ok = true;
        for (int t = first; t < total && ok; t += step) {
            const Tile w = tile_at<MODE, CG>(c, s.start, s.tiles, t, nt, tile_cols, rank, part, split);
            for (int k = w.k0; k < w.k1; k += BK, ++n) {
                const int i = n % STAGES;
                ok = __all_sync(FULL_MASK, mbar_wait(smem_u32(&s.empty[i]), ((n / STAGES) & 1) ^ 1, gave_up));
                if (!ok) break;
                if (tid == 0) *loaded = n + 1;
                load_slice<MODE, GATED>(c, w, ring + i * L::STAGE, k, wide, tid);
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&s.full[i]));
            }
        }
    } else if (MODE == WGRAD && warp >= 2 + EPI_WARPS) {
        if (c.epi.g_bias != nullptr || c.epi.g_bias_f32 != nullptr)
            for (int t = first; t < total; t += step) {
                const Tile w = tile_at<MODE, CG>(c, s.start, s.tiles, t, nt, tile_cols, rank, part, split);
                if (w.c0 == 0) {
                    const int tid = threadIdx.x - 64 - 32 * EPI_WARPS;
                    const float sum = column_sum(c, w, s.sums, tid);
                    if (split == 1)
                        put_bias_grad(c, w, tid, sum);
                    else
                        s.sum[tid] = sum;
                    __syncwarp();
                }
            }
    } else if (warp >= 2) {
        const int quad = warp & 3;            // the TMEM lanes this warp can read
        const int half = (warp - 2) >> 2;     // and its half of the columns
        WarpWriter out = {ring + RING_BYTES + (warp - 2) * STAGING, stores, lane, 0};
        if (MODE != WGRAD && c.epi.zero_rest)
            zero_rest(c.epi, s.start[0], s.start[c.E], c.R, blockIdx.x * (32 * EPI_WARPS) + threadIdx.x - 64,
                      static_cast<int64_t>(gridDim.x) * (32 * EPI_WARPS));
        uint32_t it = 0;
        for (int t = first; t < total; t += step) {
            const Tile w = tile_at<MODE, CG>(c, s.start, s.tiles, t, nt, tile_cols, rank, part, split);
            const bool any = w.k0 < w.k1;   // products were made
            if (MODE == WGRAD && !any && c.epi.add && split == 1) continue;   // nothing to add
            const int acc = it & 1;
            if (any) {
                // Should the wait be given up, the results are flagged as invalid and
                // the loop goes on, so that every warp meets the others.
                (void)mbar_wait(smem_u32(&s.acc_full[acc]), (it >> 1) & 1, gave_up, loaded);
                __syncwarp();
                tc_fence_after();
            }
            const int j0 = half * (tile_cols / 2), j1 = j0 + tile_cols / 2;
            const uint32_t d = tmem + acc * BN + (static_cast<uint32_t>(quad * 32) << 16);
            for (int j = j0; j < j1; j += EPI_COLS) {
                if (w.c0 + j >= c.epi.cols) break;
                float z[EPI_COLS], u[EPI_COLS];
                if (any) {
                    tmem_load32(d + j, z);
                    if (GATED) tmem_load32(d + wide / 2 + j, u);
                    tmem_load_wait();
                } else {
#pragma unroll
                    for (int i = 0; i < EPI_COLS; ++i) z[i] = u[i] = 0.0f;
                }
                if (split == 1) {
                    finish<MODE, GATED>(c, out, w, quad, j, z, u);
                } else {   // the ring is idle: all of this CTA's products are done
                    float4 *to = reinterpret_cast<float4 *>(ring) + ((quad * 32 + lane) * JOIN_PITCH + j) / 4;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        to[i] = make_float4(z[4 * i], z[4 * i + 1], z[4 * i + 2], z[4 * i + 3]);
                        if (GATED) to[i + BN / 8] = make_float4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
                    }
                }
                __syncwarp();
            }
            if (any) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (CG == 1)
                        mbar_arrive(smem_u32(&s.acc_empty[acc]));
                    else
                        mbar_arrive_cluster(at_rank(smem_u32(&s.acc_empty[acc]), 0));
                }
                ++it;
            }
        }
        if (split == 1 && lane == 0) tma_store_done();
    }
    __syncwarp();
    if (CG == 1 && split > 1) {   // one tile a cluster: its parts are joined
        cluster_sync();
        if (first < total) {
            const Tile w = tile_at<MODE, CG>(c, s.start, s.tiles, first, nt, tile_cols, rank, part, split);
            if (warp >= 2 && warp < 2 + EPI_WARPS) {
                WarpWriter out = {ring + RING_BYTES + (warp - 2) * STAGING, stores, lane, 0};
                for (int q = (warp - 2) * split + part; q < 4 * (tile_cols / EPI_COLS); q += EPI_WARPS * split) {
                    const int quad = q & 3, j = (q >> 2) * EPI_COLS;
                    if (w.c0 + j >= c.epi.cols) continue;
                    const uint32_t at = smem_u32(ring) + (quad * 32 * JOIN_PITCH + j) * 4;
                    float *turn = reinterpret_cast<float *>(ring + JOIN_BYTES + (warp - 2) * TURN_BYTES);
                    float z[EPI_COLS], u[EPI_COLS];
                    join32(at, split, turn, lane, z);
                    if (GATED) join32(at + BN / 2 * 4, split, turn, lane, u);
                    finish<MODE, GATED>(c, out, w, quad, j, z, u);
                    __syncwarp();
                }
                if (lane == 0) tma_store_done();
            } else if (MODE == WGRAD && warp >= 2 + EPI_WARPS && part == 0 && w.c0 == 0 &&
                       (c.epi.g_bias != nullptr || c.epi.g_bias_f32 != nullptr)) {
                const int tid = threadIdx.x - 64 - 32 * EPI_WARPS;
                float t = 0.0f;
                for (int r = 0; r < split; ++r) t += peer_float(at_rank(smem_u32(&s.sum[tid]), r));
                put_bias_grad(c, w, tid, t);
            }
        }
        __syncwarp();
        cluster_sync();   // peers have read this CTA's part
    }
    tc_fence_before();
    if (CG == 2)
        cluster_sync();   // the pair's products and arrivals are done
    else
        __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_free<CG>(tmem, TMEM_COLS);
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

// Clusters of `size` CTAs that the device holds at once; the same for all these
// kernels, one CTA to an SM.
template <typename K> int cluster_count(K kernel, int threads, int size)
{
    static std::atomic<int> known[64][9];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 1;
    if (dev < 64 && (n = known[dev][size].load(std::memory_order_relaxed)) > 0) return n;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = size;
    cfg.blockDim = threads;
    cfg.dynamicSmemBytes = TC_SMEM;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
        (void)cudaGetLastError();
        n = sm_count() / (2 * size) + 1;
    }
    if (dev < 64) known[dev][size].store(n, std::memory_order_relaxed);
    return n;
}

// Cycles that the load warps take for a row of a slice.
constexpr int RAW_ROW = 15;

// How a call is cut: columns of a tile (both parts of a gated one), CTAs a tile's
// contraction is split over.
struct Cut {
    int wide, split;
};

template <int MODE> int64_t tile_rows(const ExpertCall &c, int high)
{
    return MODE == WGRAD ? static_cast<int64_t>(c.E) * ((c.N + high - 1) / high) : c.R / high + (c.R < c.E ? c.R : c.E);
}

// Single CTAs: the cut that is done first by a count of cycles, fitted to 27 calls
// measured with all cuts (on 36 others it took the best cut or one at most 9% slower).
// A slice takes its bytes at 64 a cycle, but 560 cycles at least with four in flight
// (RAW_ROW a row where the load warps read it); a tile's epilogue overlaps the
// next tile's products; a join grows with its parts.  An expert has half a tile more
// than its rows fill, and one at least.  us with 256 columns unsplit, and as cut: 300 rows by 3 experts of
// 1,000 x 1,000 14.4, 9.1 (64); x 4,000 23.3, 15.8 (192 in 4 parts); 2,999 rows by
// 40 of 1,009 x 1,000 26.9, 23.9 (192); 500 rows by one of 512 x 8,192 42, 16.7 (64 in 4);
// weight gradients of 2,000 rows, 512 x 1,024 16.5, 12.3 (128 in 4), of 21,063 rows,
// 112 x 1,624 164, 27.7 (128 in 8).
template <int MODE, bool GATED> Cut choose_cut(const ExpertCall &c, bool raw)
{
    const int64_t depth = MODE == FWD ? c.K : MODE == DGRAD ? c.N : c.R / c.E, slices = (depth + BK - 1) / BK;
    const int64_t some = c.R < c.E ? c.R : c.E, filled = c.R / BM + some / 2;
    const int64_t high = MODE == WGRAD ? tile_rows<MODE>(c, BM) : filled > some ? filled : some;
    const int sms = sm_count();
    Cut best = {BN, 1};
    int64_t least = INT64_MAX;
    for (int wide = BN; wide >= (GATED ? 128 : 64); wide -= GATED ? 128 : 64) {
        const int cols = GATED ? wide / 2 : wide;
        const int64_t nt = (c.epi.cols + cols - 1) / cols, tiles = nt * tile_rows<MODE>(c, BM);
        for (int split = 1; split <= 8; split *= 2) {
            if (split > 1 && (tiles * split > sms ||
                              tiles > cluster_count(k_expert_tc<MODE, GATED, 1, true>, tc_threads(MODE, false), split)))
                break;
            const int64_t waves = split > 1 ? 1 : (nt * high + sms - 1) / sms;
            const int64_t by_tma = 256 + 2 * wide > 560 ? 256 + 2 * wide : 560;
            const int64_t slice = raw ? RAW_ROW * (BM + wide) : by_tma, epilogue = 1500 + 14 * wide;
            const int64_t part = (slices + split - 1) / split * slice;
            const int64_t cycles = waves * (part > epilogue ? part : epilogue) + epilogue +
                                   (split > 1 ? 3500 + 1000 * split : 0);
            if (cycles < least) {
                least = cycles;
                best = Cut{wide, split};
            }
        }
    }
    return best;
}

template <int MODE, bool GATED, int CG, bool ANY, bool RAW = false>
mp_status_t launch_tc(const ExpertCall &c, const CUtensorMap &a, const CUtensorMap &b, const StoreMaps &m, Cut cut)
{
    static std::atomic<uint64_t> allowed{0};
    if (!allow_smem(k_expert_tc<MODE, GATED, CG, ANY, RAW>, allowed, TC_SMEM)) return MP_ERR_CUDA;
    const int cols = GATED ? cut.wide / 2 : cut.wide, split = cut.split;
    const int64_t tiles = (c.epi.cols + cols - 1) / cols * tile_rows<MODE>(c, CG * BM);
    if (tiles > INT32_MAX / 2) return MP_ERR_UNSUPPORTED;   // counted in 32 bits
    const int64_t room = CG == 1 ? sm_count() : cluster_count(k_expert_tc<MODE, GATED, CG, ANY, RAW>, tc_threads(MODE, RAW), 2);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = static_cast<unsigned>(split > 1 ? split * tiles : CG * (tiles < room ? tiles : room));
    cfg.blockDim = tc_threads(MODE, RAW);
    cfg.dynamicSmemBytes = TC_SMEM;
    cfg.stream = c.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CG * split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CG * split == 1 ? 1 : 2;
    (void)cudaLaunchKernelEx(&cfg, k_expert_tc<MODE, GATED, CG, ANY, RAW>, a, b, m, c, split, cut.wide);
    return check_launch();
}

// Whether pairs of CTAs take the call.  A pair reads a third less per product from
// L2, which bounds the single CTAs: 131,072 x 4,096 rows by 128 experts of 2,048
// 1,377 -> 1,211 us; weight gradients of 8 x 2,048 rows, 4,096 x 4,096, 370 -> 344.
// But its tile has 256 rows, of which an expert leaves half of one empty on average,
// and the hand-over of the accumulator between the CTAs counts where the contraction
// is short.  us of single CTAs / pairs, 64 experts, one in eight empty (the bits are the same):
//   rows an expert            256      320      384      512      1,024
//   2,048 x 2,048           143/134  148/148  172/161  209/201  375/346
//   its row gradient        147/129  151/147  176/160  228/212  440/390
// With loads all equal, 384 rows fill a tile and a half: 168/178 and 177/184, 512 rows
// 213/186 and 221/189.  The border, 384, lies between the two.
//   contraction of            512      640      768      896     1,024
//   384 rows, 2,048 wide     57/67    66/71    76/73    85/82    94/91
//   row gradient             61/66    70/65    80/70      -      98/91
//   1,024 rows, 2,048 wide  119/133  140/140  160/148  182/166  205/190
//   row gradient            129/124  154/132  173/145     -     217/186
// From 768 (row gradients 640) on neither loses.  Weight gradients, whose contraction is the rows (2,048 x
// 2,048): 384 rows 199/208, 512 rows 239/238 (equal loads 233/219), 1,024 rows 418/413
// (408/389).
// With fewer tiles than SMs another cut does more (choose_cut).
template <int MODE> bool in_pairs(const ExpertCall &c)
{
    const int64_t cols = act_gated(c.epi.act) && MODE == FWD ? 2ll * c.epi.cols : c.epi.cols;
    const int depth = MODE == FWD ? c.K : c.N;   // of the products of rows
    return c.R >= (MODE == WGRAD ? 512 : 384) * static_cast<int64_t>(c.E) &&
           (MODE == WGRAD || depth >= (MODE == FWD ? 768 : 640)) &&
           (cols + BN - 1) / BN * (MODE == WGRAD ? static_cast<int64_t>(c.E) * ((c.N + BM - 1) / BM) : c.R / BM) >= sm_count();
}

// Whether TMA can address the operands.
template <int MODE> bool by_tma(const ExpertCall &c)
{
    return c.R > 0 && c.K % 8 == 0 && (MODE == FWD || c.N % 8 == 0) && aligned16(c.a) && aligned16(c.b);
}

template <int MODE, bool GATED> mp_status_t cut_and_launch(const ExpertCall &c)
{
    const bool raw = !by_tma<MODE>(c), pairs = !raw && in_pairs<MODE>(c);
    static std::atomic<uint64_t> allowed{0};
    if (!allow_smem(k_expert_tc<MODE, GATED, 1, true>, allowed, TC_SMEM)) return MP_ERR_CUDA;
    const Cut cut = pairs ? Cut{BN, 1} : choose_cut<MODE, GATED>(c, raw);
    CUtensorMap a = {}, b = {};
    const uint64_t R = c.R, N = c.N, K = c.K, E = c.E;
    const uint64_t da[2] = {MODE == FWD ? K : N, R};
    const uint32_t box_a[2] = {64, MODE == WGRAD ? 64u : static_cast<uint32_t>(BM)};
    const uint64_t db[3] = {K, MODE == WGRAD ? R : N, E};
    const uint32_t box_b[3] = {64, MODE == FWD ? cut.wide / 2u : 64u, 1};
    if (!raw && (!make_map(&a, c.a, 2, da, box_a) || !make_map(&b, c.b, MODE == WGRAD ? 2 : 3, db, box_b))) {
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
    if (raw) return launch_tc<MODE, GATED, 1, true, true>(c, a, b, m, cut);
    if (pairs) return launch_tc<MODE, GATED, 2, false>(c, a, b, m, cut);
    if (MODE == WGRAD && cut.wide == BN) return launch_tc<MODE, GATED, 1, MODE != WGRAD>(c, a, b, m, cut);
    return launch_tc<MODE, GATED, 1, true>(c, a, b, m, cut);
}

}  // namespace

template <int MODE> mp_status_t expert_tc(const ExpertCall &c)
{
    if (MODE == FWD && act_gated(c.epi.act)) return cut_and_launch<MODE, MODE == FWD>(c);
    return cut_and_launch<MODE, false>(c);
}

bool expert_by_tma(const ExpertCall &c, int mode)
{
    return mode == FWD ? by_tma<FWD>(c) : by_tma<DGRAD>(c);   // WGRAD reads the columns DGRAD does
}

template mp_status_t expert_tc<FWD>(const ExpertCall &);
template mp_status_t expert_tc<DGRAD>(const ExpertCall &);
template mp_status_t expert_tc<WGRAD>(const ExpertCall &);

}  // namespace mp
