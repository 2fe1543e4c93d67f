// What the norms before and after a block and their gradients share: how a row lies
// over threads, its way through shared memory, and sums over it.
//
// Bytes bound these operators: a row is read once, worked on in registers, and written once.
// W threads own a row, 16 values each, and a CTA of up to 512 threads works on R rows at a
// time, each a group of its own with a barrier of its own.  While a group works on a row, its
// next ones are on their way into shared memory, in as many slots as there is room for.  What
// counts next is instructions: 8 values a thread took 81 a value (two norms, 4,096 wide: 188
// us, the issue slots 81% full); hence 16, and arithmetic on pairs of fp32 (fma.rn.f32x2).
//   ROWS_BULK  rows of whole 16-byte vectors on 16-byte boundaries, 2 KB or more: one bulk copy a
//              row and tensor (gradient at one norm, 16,384 x 4,096, alone: 88 us, by cp.async 96).
//   ROWS_VEC   shorter ones: a thread copies vectors tid, tid + W, ... of the row by cp.async
//              and reads nobody else's.
//   ROWS_ANY   rows that start anywhere: the group copies the 16-byte granules that hold the row,
//              and lane l of a warp reads values l, l + 32, ... of the warp's run of 512; a barrier
//              in between.  All but a row's last warp have a whole run and ask nothing for each value.
//   ROWS_NARROW  such rows of up to 256 values, several a warp: values tid, tid + W, ...
//   C 4      rows of more than 8192 values, and fp32 gradients of which one row and the sums beside it are more than
//            shared memory (both norms: from 6,145 wide with biases, 5,633 with a gate for each value too, 5,121 with
//            one for each channel): not staged, the threads read them as they need them.  That costs gradients most
//            (4,096 x 7,168 fp32, layer norms with biases: 1,230 us, floor 105; 4,096 x 6,144, staged: 171, floor 90).
#pragma once

#include <cuda_fp16.h>

#include <type_traits>

#include "pairs.cuh"
#include "tc.cuh"

namespace mp {

constexpr int NORM_SHARED = 5;      // gradients shared by rows: two weights, two biases, the gate
constexpr int NORM_PARTS = 152;     // partial sums of each at most: a CTA an SM
constexpr int NORM_THREADS = 512;   // of a CTA, C 4: twice as many
constexpr int NORM_BUDGET = 112 * 1024;   // shared memory of one of two CTAs on an SM
constexpr int NORM_MOST = 225 * 1024;     // of one alone
constexpr int NORM_SLOTS = 4;

enum { ROWS_ANY, ROWS_NARROW, ROWS_VEC, ROWS_BULK };

// How T rows of H values are laid out.
struct NormPlan {
    int W, R;         // threads a row, rows a CTA at a time
    int stages, pitch;   // slots of a group, bytes of one tensor's row in a slot
    int held;            // bytes of a vector that the rows share
    size_t smem;
};

struct NormRows {
    const void *at;   // [T,H]
    int64_t end;      // address past its last byte
};
// The tensors whose rows go through shared memory, and a row's place in a slot (-1: absent).
struct NormInputs {
    NormRows rows[5];
    int slot[5], tensors;
    void add(int i, const NormRows &r) { rows[i] = r; slot[i] = r.at != nullptr ? tensors++ : -1; }
};

__device__ __forceinline__ float norm_value(float v) { return v; }
__device__ __forceinline__ float norm_value(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float norm_value(__half v) { return __half2float(v); }
__device__ __forceinline__ void norm_put(float *p, float v) { *p = v; }
__device__ __forceinline__ void norm_put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void norm_put(__half *p, float v) { *p = __float2half_rn(v); }

// The values of a 16-byte vector, in pairs.
__device__ __forceinline__ void vec_values(const uint4 &v, f2 *f, const __nv_bfloat16 *)
{
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = pair(bf16_lo(u[i]), bf16_hi(u[i]));
}
__device__ __forceinline__ void vec_values(const uint4 &v, f2 *f, const __half *)
{
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(u + i));
        f[i] = pair(t.x, t.y);
    }
}
__device__ __forceinline__ void vec_values(const uint4 &v, f2 *f, const float *)
{
    f[0] = pair(__uint_as_float(v.x), __uint_as_float(v.y));
    f[1] = pair(__uint_as_float(v.z), __uint_as_float(v.w));
}
__device__ __forceinline__ uint32_t two_of(f2 v, const __nv_bfloat16 *)
{
    const float2 r = both(v);
    return pack_bf16x2(r.x, r.y);
}
__device__ __forceinline__ uint32_t two_of(f2 v, const __half *)
{
    const float2 r = both(v);
    const __half2 h = __floats2half2_rn(r.x, r.y);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <typename D> __device__ __forceinline__ uint4 vec_of(const f2 *f, const D *p)
{
    return make_uint4(two_of(f[0], p), two_of(f[1], p), two_of(f[2], p), two_of(f[3], p));
}
__device__ __forceinline__ uint4 vec_of(const f2 *f, const float *)
{
    const float2 a = both(f[0]), b = both(f[1]);
    return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes = 16)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the last `left` groups of this thread have landed.
__device__ __forceinline__ void cp_wait(int left)
{
    switch (left) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    }
}

// One group's view of its rows: N values a thread, in N2 pairs.
template <typename D, int M, int C> struct NormGroup {
    static constexpr bool VEC = M == ROWS_VEC || M == ROWS_BULK;
    static constexpr int N = 8 * C, N2 = 4 * C;
    static constexpr int NV = 16 / sizeof(D);    // values a vector
    static constexpr int VECS = N / NV;
    static constexpr bool STAGED = C < 4;
    static constexpr int WARPS = 32;   // of a row at most
    static constexpr bool RUNS = M == ROWS_ANY;   // a warp's values lie side by side
    static constexpr int RUN = 32 * N;            // of a warp

    int W, H, tid, group;
    float *red;           // [2][M_MOST][WARPS] of this group: see sums()
    uint32_t bars;        // ROWS_BULK: an mbarrier for each slot
    volatile int *gave_up;
    int phase = 0;
    uint32_t slot_phase = 0;

    // What comes first in shared memory: the groups' sums, their mbarriers, a flag.  (Groups of
    // less than a warp need neither of the first.)
    static constexpr int RED = 2 * 3 * 32;   // floats a group
    static constexpr __host__ __device__ size_t head(int W, int R) { return (W < 32 ? 1 : R) * (RED * 4 + NORM_SLOTS * 8) + 16; }
    __device__ __forceinline__ void begin(uint8_t *smem, int W_, int R, int H_)
    {
        W = W_;
        H = H_;
        group = threadIdx.x / W;
        tid = threadIdx.x - group * W;
        const int own = W < 32 ? 0 : group;
        red = reinterpret_cast<float *>(smem) + own * RED;
        for (int i = tid; i < RED; i += W) red[i] = 0.0f;
        bars = smem_u32(smem + (W < 32 ? 1 : R) * RED * 4 + own * NORM_SLOTS * 8);
        int *const flag = reinterpret_cast<int *>(smem + head(W, R) - 16);
        gave_up = flag;
        if (M == ROWS_BULK && tid == 0) {
            for (int i = 0; i < NORM_SLOTS; ++i) mbar_init(bars + 8 * i, 1);
            mbar_init_fence();
        }
        if (threadIdx.x == 0) *flag = 0;
        __syncthreads();
    }

    __device__ __forceinline__ void barrier() const
    {
        __syncwarp();   // a warp comes to the barrier as a whole
        if (W > 32)
            asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(W) : "memory");
    }

    // The sums over the row, each added up in a fixed order; every thread gets them.  A
    // warp's lanes first (W <= 32: the W lanes of the row), then the warps.  Two
    // buffers in turn: a thread that is still reading one is waited for by the barrier
    // of the next sum.
    template <int S> __device__ __forceinline__ void sums(float (&v)[S])
    {
#pragma unroll
        for (int d = 16; d; d >>= 1)
            if (d < W) {
#pragma unroll
                for (int i = 0; i < S; ++i) v[i] += __shfl_xor_sync(FULL_MASK, v[i], d);
            }
        if (W <= 32) return;
        float *to = red + (phase & 1) * M_MOST * WARPS;
        phase ^= 1;
        if ((threadIdx.x & 31) == 0) {
#pragma unroll
            for (int i = 0; i < S; ++i) to[i * WARPS + (tid >> 5)] = v[i];
        }
        barrier();
        const int warps = W >> 5;   // slots past the last warp hold 0
        if (warps <= 8) {
#pragma unroll
            for (int i = 0; i < S; ++i) {
                const float4 p = reinterpret_cast<const float4 *>(to + i * WARPS)[0];
                const float4 q = reinterpret_cast<const float4 *>(to + i * WARPS)[1];
                v[i] = ((p.x + p.y) + (p.z + p.w)) + ((q.x + q.y) + (q.z + q.w));
            }
        } else {
#pragma unroll
            for (int i = 0; i < S; ++i) v[i] = to[i * WARPS + (threadIdx.x & 31)];
#pragma unroll
            for (int d = 16; d; d >>= 1) {
#pragma unroll
                for (int i = 0; i < S; ++i) v[i] += __shfl_xor_sync(FULL_MASK, v[i], d);
            }
        }
    }
    static constexpr int M_MOST = 3;

    // Column of pair i; the second of the pair is `beside` further on.
    __host__ __device__ __forceinline__ int col(int i) const
    {
        return VEC ? (2 * i / NV * W + tid) * NV + 2 * i % NV : first() + step(i);
    }
    __host__ __device__ __forceinline__ int step(int i) const { return RUNS ? 64 * i : 2 * i * W; }
    __host__ __device__ __forceinline__ int beside() const { return VEC ? 1 : RUNS ? 32 : W; }
    __host__ __device__ __forceinline__ int first() const { return RUNS ? (tid >> 5) * RUN + (tid & 31) : tid; }
    // Whether the row has all of this warp's run: then nothing is asked for each value.
    __device__ __forceinline__ bool whole() const { return (tid >> 5) * RUN + RUN <= H; }

    // Values of a row (or of what is shared by the rows) at `p`, 0 past its end.
    __device__ __forceinline__ void load(const D *p, f2 (&f)[N2]) const
    {
        if (VEC) {
#pragma unroll
            for (int v = 0; v < VECS; ++v) {
                const int at = (v * W + tid) * NV;
                uint4 u = make_uint4(0, 0, 0, 0);
                if (at < H) u = *reinterpret_cast<const uint4 *>(p + at);
                vec_values(u, f + v * (NV / 2), p);
            }
        } else if (RUNS && whole()) {
            const D *const from = p + first();
#pragma unroll
            for (int i = 0; i < N2; ++i) f[i] = pair(norm_value(from[64 * i]), norm_value(from[64 * i + 32]));
        } else {
            const D *const from = p + first();
            const int left = H - first();
#pragma unroll
            for (int i = 0; i < N2; ++i) {
                const int at = step(i), next = at + beside();
                f[i] = pair(at < left ? norm_value(from[at]) : 0.0f, next < left ? norm_value(from[next]) : 0.0f);
            }
        }
    }
    // The same of what hold() has copied (STAGED; else of where it is).
    __device__ __forceinline__ void load_shared(const D *p, f2 (&f)[N2]) const
    {
        if (RUNS && STAGED) {
            const D *const from = p + first();
#pragma unroll
            for (int i = 0; i < N2; ++i) f[i] = pair(norm_value(from[64 * i]), norm_value(from[64 * i + 32]));
        } else {
            load(p, f);
        }
    }
    __device__ __forceinline__ void store(D *p, const f2 (&f)[N2]) const
    {
        if (VEC) {
#pragma unroll
            for (int v = 0; v < VECS; ++v) {
                const int at = (v * W + tid) * NV;
                if (at < H) *reinterpret_cast<uint4 *>(p + at) = vec_of(f + v * (NV / 2), p);
            }
        } else if (RUNS && whole()) {
            D *const to = p + first();
#pragma unroll
            for (int i = 0; i < N2; ++i) {
                const float2 r = both(f[i]);
                norm_put(to + 64 * i, r.x);
                norm_put(to + 64 * i + 32, r.y);
            }
        } else {
            D *const to = p + first();
            const int left = H - first();
#pragma unroll
            for (int i = 0; i < N2; ++i) {
                const int at = step(i), next = at + beside();
                const float2 r = both(f[i]);
                if (at < left) norm_put(to + at, r.x);
                if (next < left) norm_put(to + next, r.y);
            }
        }
    }
    // Sums of the rows' values in shared memory, [N2][W] pairs, each thread's its own: banks are
    // used evenly, and what is past the row's end adds 0.  (In the order of the columns, eight
    // threads to a bank, two biases took 2/3 of a gradient's time.)
    __device__ __forceinline__ void pile(f2 *p, const f2 (&f)[N2]) const
    {
#pragma unroll
        for (int i = 0; i < N2; ++i) p[i * W + tid] = add2(p[i * W + tid], f[i]);
    }
    // The sum of column c there.
    __device__ __forceinline__ float piled(const f2 *p, int c) const
    {
        int i, t, second;
        if (VEC) {
            const int v = c / NV, e = c % NV;
            i = v / W * (NV / 2) + (e >> 1); t = v % W; second = e & 1;
        } else {
            const int k = RUNS ? (c % RUN) >> 5 : c / W;
            i = k >> 1; t = RUNS ? c / RUN * 32 + (c & 31) : c % W; second = k & 1;
        }
        return reinterpret_cast<const float *>(p + i * W + t)[second];
    }
    // fp32 sums a column: set, or added to.
    template <bool ADD> __device__ __forceinline__ void columns(float *p, const f2 (&f)[N2]) const
    {
#pragma unroll
        for (int i = 0; i < N2; ++i) {
            const int at = col(i), next = at + beside();
            const float2 r = both(f[i]);
            if (at < H) p[at] = ADD ? p[at] + r.x : r.x;
            if (next < H) p[next] = ADD ? p[next] + r.y : r.y;
        }
    }
    // Pair i with 0 in the place of what is past the row's end.
    __device__ __forceinline__ f2 inside(int i, f2 v) const
    {
        if (VEC) return col(i) < H ? v : 0ull;
        const float2 r = both(v);
        return pair(col(i) < H ? r.x : 0.0f, col(i) + beside() < H ? r.y : 0.0f);
    }

    // Starts the copy of row t of `rows` into `slot`, by cp.async.
    __device__ __forceinline__ void fetch_one(const NormRows &rows, uint32_t t, uint8_t *slot) const
    {
        if (!STAGED) return;
        const char *row = static_cast<const char *>(rows.at) + static_cast<uint64_t>(t) * (H * static_cast<uint32_t>(sizeof(D)));
        const uint32_t to = smem_u32(slot);
        if (VEC) {
#pragma unroll
            for (int v = 0; v < VECS; ++v) {
                const int at = (v * W + tid) * 16;
                if (at < H * static_cast<int>(sizeof(D))) cp_async16(to + at, row + at);
            }
        } else {
            const int off = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15u);
            const int granules = (off + H * static_cast<int>(sizeof(D)) + 15) / 16;
            const char *from = row - off;
            if (from >= static_cast<const char *>(rows.at) && reinterpret_cast<int64_t>(from) + granules * 16 <= rows.end) {
                from += tid * 16;   // not the tensor's first or last row: nothing is asked for each granule
                uint32_t dst = to + tid * 16;
#pragma unroll 1
                for (int q = tid; q < granules; q += W, from += W * 16, dst += W * 16) cp_async16(dst, from);
                return;
            }
#pragma unroll 1
            for (int q = tid; q < granules; q += W) {
                const char *src = row - off + q * 16;
                const int64_t left = rows.end - reinterpret_cast<int64_t>(src);
                if (src >= static_cast<const char *>(rows.at)) {
                    cp_async16(to + q * 16, src, left < 16 ? static_cast<int>(left) : 16);
                } else {   // the granule begins before the tensor: only what is of it is read
                    for (int i = off; i < 16 && i < off + H * static_cast<int>(sizeof(D)); i += sizeof(D))
                        *reinterpret_cast<D *>(slot + i) = *reinterpret_cast<const D *>(src + i);
                }
            }
        }
    }
    // Starts the copy of row t, if there is one, into slot `i` at `slot`.  Where this is done in several
    // places the tensors are a loop (U 1): copies of granules are much code, and gradients of rows
    // that start anywhere wait for instructions (4,099 x 4,097 143 -> 128 us).
    template <int U>
    __device__ __forceinline__ void fetch(const NormInputs &in, uint32_t t, uint32_t T, uint8_t *slot, int pitch, int i) const
    {
        if (!STAGED) return;
        if (M != ROWS_VEC && W <= 32) __syncwarp();   // the warp has read the slot, where no barrier says so
        if (M == ROWS_BULK) {
            if (tid != 0 || t >= T) return;
            if (*gave_up) return;   // a slot whose row has not come takes no other
            const uint32_t bytes = static_cast<uint32_t>(H) * sizeof(D);
            mbar_expect(bars + 8 * i, bytes * in.tensors);
#pragma unroll
            for (int k = 0; k < 5; ++k)
                if (in.slot[k] >= 0)
                    bulk_load(smem_u32(slot) + in.slot[k] * pitch,
                              static_cast<const char *>(in.rows[k].at) + static_cast<uint64_t>(t) * bytes, bytes, bars + 8 * i);
        } else {
            if (t < T) {
#pragma unroll(VEC ? 5 : U)
                for (int k = 0; k < 5; ++k)
                    if (in.slot[k] >= 0) fetch_one(in.rows[k], t, slot + in.slot[k] * pitch);
            }
            cp_commit();
        }
    }
    // Waits for the row in slot i of `slots`; `there`: whether there is one.
    __device__ __forceinline__ void arrived(int i, int slots, bool there) const
    {
        if (!STAGED) return;
        if (M == ROWS_BULK) {
            if (there) (void)mbar_wait(bars + 8 * i, slot_phase, gave_up);
        } else {
            cp_wait(slots - 1);
            if (!VEC) barrier();
        }
    }
    // The slot after slot i.
    __device__ __forceinline__ int after(int i, int slots)
    {
        if (i + 1 < slots) return i + 1;
        slot_phase ^= 1u;
        return 0;
    }
    // At the end, in front of slot i: no copy is left in flight.  After a wait given up thread 0 has started no more of
    // them (fetch), the rows that were left have gone by as the slots were, since all threads have to come to the
    // barriers, and each slot's phase at hand is waited for here, whichever of the two it is; where nothing is on its way
    // that is 1 s.  (A verdict on each row, by which its results are not stored and the loop is left, makes a row's loads
    // wait for it: the gradient at both norms, 32,768 x 7,168, took 639 to 770 us with one in place of 603, the norm of
    // 16,384 x 4,096 88 to 94 in place of 87.)
    __device__ __forceinline__ void finish(int i, int slots, int32_t *status) const
    {
        if (!STAGED) return;
        if (M != ROWS_BULK) {
            cp_wait(0);
        } else if (*gave_up && tid == 0) {
            for (int k = 0; k < slots; ++k) {
                const uint32_t last = k < i ? slot_phase : slot_phase ^ 1u;
                mbar_drain(bars + 8 * k, last);
                mbar_drain(bars + 8 * k, last ^ 1u);
            }
            or_status(status, MP_STATUS_STALLED);
        }
    }
    // What the rows share, copied to `to` by the whole CTA: there after finish_held() and a barrier.
    __device__ __forceinline__ void hold(const D *from, uint8_t *to) const
    {
        if (VEC) {
            for (int c = threadIdx.x; c < H / NV; c += blockDim.x) cp_async16(smem_u32(to) + c * 16, from + c * NV);
        } else {
            const int end = RUNS ? W * N : H;   // to the end of the last warp's run: 0
            for (int c = threadIdx.x; c < end; c += blockDim.x) norm_put(reinterpret_cast<D *>(to) + c, c < H ? norm_value(from[c]) : 0.0f);
        }
    }

    // Where row t of `rows` can be read: in `slot`, or where it is.
    __device__ __forceinline__ const D *row(const NormRows &rows, uint32_t t, const uint8_t *slot) const
    {
        if constexpr (STAGED && VEC) {
            return reinterpret_cast<const D *>(slot);
        } else {
            const D *at = static_cast<const D *>(rows.at) + static_cast<uint64_t>(t) * static_cast<uint32_t>(H);
            if constexpr (STAGED)
                return reinterpret_cast<const D *>(slot + (reinterpret_cast<uintptr_t>(at) & 15u));
            else
                return at;
        }
    }
};

// Columns of a group's fp32 sums, to whole 16 bytes.
__host__ __device__ inline int norm_wide(int H) { return (H + 3) / 4 * 4; }

// Threads a row, rows at a time, and slots for `tensors` staged rows; `held` vectors that the
// rows share lie beside them, and `sums` of the rows' values of each group.  Two CTAs on an SM wherever two slots or more fit in half of it.
template <typename D> NormPlan norm_plan(int64_t T, int H, int C, int threads, int form, int tensors, int held, int sums, bool two)
{
    NormPlan p;
    const int need = (H + 8 * C - 1) / (8 * C);
    p.W = 1;
    if (need <= 32)
        while (p.W < need) p.W *= 2;
    else
        p.W = (need + 31) / 32 * 32;
    p.R = C < 4 ? threads / p.W : 1;
    while (p.R > 1 && p.W * (p.R / 2) >= 32 && (T + p.R / 2 - 1) / (p.R / 2) <= sm_count()) p.R /= 2;   // few rows: spread
    p.pitch = (H * static_cast<int>(sizeof(D)) + 15) / 16 * 16 + 16;
    const bool bulk = form == ROWS_BULK;
    const int runs = p.W * 8 * C * static_cast<int>(sizeof(D));   // what the warps' runs take
    p.held = form == ROWS_ANY && runs > p.pitch ? runs : p.pitch;
    size_t fixed, slot;
    for (;; p.R = p.W < 32 ? p.R / 2 : p.R - 1) {
        const int64_t extra = C < 4 ? static_cast<int64_t>(held) * p.held + static_cast<int64_t>(sums) * p.R * p.W * 32 * C : 0;
        fixed = NormGroup<D, ROWS_ANY, 2>::head(p.W, p.R) + static_cast<size_t>(extra);
        slot = static_cast<size_t>(p.pitch) * tensors * p.R;
        p.stages = 0;
        if (C < 4) {
            const size_t room = two && fixed + 2 * slot <= NORM_BUDGET ? NORM_BUDGET : NORM_MOST;
            p.stages = fixed < room ? static_cast<int>((room - fixed) / slot) : 0;
            if (p.stages > (bulk ? 3 : NORM_SLOTS)) p.stages = bulk ? 3 : NORM_SLOTS;   // of bulk copies more are slower (88.6, 88.7, 90.7 us with 2, 3, 4)
        }
        // Fewer rows at a time rather than none on their way, where bytes count (gradients at both norms,
        // fp32: 2,048 x 2,048 26.8 -> 23.8 us); rows that start anywhere are bound by instructions (2,047 x
        // 2,050 42.9 -> 48.6) and only have to fit.  A CTA stays whole warps; rows of less than a warp always fit.
        if (p.stages >= (bulk ? 2 : 1) || p.R == 1 || p.W * p.R <= 32) break;
    }
    const int64_t steps = (T + p.R - 1) / p.R;
    if (p.stages > steps) p.stages = static_cast<int>(steps);
    p.smem = fixed + slot * p.stages;
    return p;
}

// How the rows of a call are staged.
template <typename D> bool norm_by_bulk(int H) { return H * static_cast<int>(sizeof(D)) >= 2048; }
inline bool norm_is_narrow(int H) { return H <= 256; }   // less than a warp's lanes of 16 values

// The launchers of the types' kernels (norm_fwd.cu, norm_bwd_*.cu).
struct NormCall {
    NormRows x, residual, gate_rows, s, g_s, g_y;   // [T,H], `at` NULL where absent
    const void *post_w, *post_b, *gate, *pre_w, *pre_b;
    int64_t T;
    int H, kind, gate_form;
    float eps, scale;
    bool vec;                  // every tensor is whole 16-byte vectors
    int32_t *status;
    void *s_out, *y;
    float *stats;
    void *g_x, *g_residual, *g_gate;
    float *sums[NORM_SHARED];  // [grid,H] or NULL: post_w, post_b, pre_w, pre_b, gate
    cudaStream_t stream;
};
template <typename D> mp_status_t norm_forward(const NormCall &c);
template <typename D> mp_status_t norm_backward(const NormCall &c, int &parts);

// Launches `kernel` over the rows.  `two`: compiled for two CTAs on an SM.
template <typename K, typename... A>
mp_status_t norm_launch(K kernel, std::atomic<uint64_t> &allowed, NormPlan p, int form, bool two, int64_t T,
                        cudaStream_t stream, int &grid, A... args)
{
    // Rows in runs belong to whole warps, and sums cross whole warps: norm_plan gives nothing else.
    if (p.W * p.R % 32 != 0 || (form == ROWS_ANY && p.W % 32 != 0)) return MP_ERR_UNSUPPORTED;
    if (!allow_smem(kernel, allowed, NORM_MOST)) return MP_ERR_CUDA;
    const int64_t steps = (T + p.R - 1) / p.R, most = sm_count() * (two && p.smem <= NORM_BUDGET ? 2 : 1);
    grid = static_cast<int>(steps < most ? steps : most);
    if (!two && grid > NORM_PARTS) grid = NORM_PARTS;   // gradients
    (void)launch_pdl(kernel, grid, p.W * p.R, p.smem, stream, args..., p);
    return check_launch();
}

}  // namespace mp
