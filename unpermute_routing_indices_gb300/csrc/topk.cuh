// Selection inside a warp, shared by the routers.
#pragma once

#include "common.cuh"

namespace mp {

// A 32-bit key with the order of the floats: key(a) < key(b) iff a < b (for
// non-NaN values; -0 and +0 get the same key).  Every float's key is > 0, so 0
// stands for "no candidate".
__device__ __forceinline__ uint32_t order_key(float f)
{
    const uint32_t u = __float_as_uint(__fadd_rn(f, 0.0f));   // -0 becomes +0
    return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t k)
{
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// Arg-max across the warp on (key desc, index asc); every lane gets the
// winning index (the key is returned through `key`).
__device__ __forceinline__ uint32_t warp_argmax_key(uint32_t &key, uint32_t idx)
{
    const uint32_t m = __reduce_max_sync(FULL_MASK, key);
    const uint32_t i = __reduce_min_sync(FULL_MASK, key == m ? idx : 0xffffffffu);
    key = m;
    return i;
}

// Compare-exchange for a descending order on (key desc, index asc).
__device__ __forceinline__ void cx_desc(uint32_t &ka, uint32_t &ia, uint32_t &kb, uint32_t &ib)
{
    const bool keep = ka > kb || (ka == kb && ia < ib);
    const uint32_t k0 = keep ? ka : kb, k1 = keep ? kb : ka;
    const uint32_t i0 = keep ? ia : ib, i1 = keep ? ib : ia;
    ka = k0; kb = k1; ia = i0; ib = i1;
}

// Batcher's odd-even merge sort of N (a power of two) (key, index) pairs,
// descending; every index is a compile-time constant once unrolled.
template <int N>
__device__ __forceinline__ void sort_desc(uint32_t (&k)[N], uint32_t (&ix)[N])
{
#pragma unroll
    for (int p = 1; p < N; p <<= 1)
#pragma unroll
        for (int q = p; q >= 1; q >>= 1)
#pragma unroll
            for (int j = q % p; j + q < N; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i)
                    if (i + j + q < N && (i + j) / (2 * p) == (i + j + q) / (2 * p))
                        cx_desc(k[i + j], ix[i + j], k[i + j + q], ix[i + j + q]);
}

}  // namespace mp
