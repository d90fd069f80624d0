// rows.h -- pieces of E consecutive elements of rows of any width and
// alignment, as fp32 (device side).
#pragma once

#include "twell_device.h"

namespace twell {

// Vectors that need the alignment of their elements only.
typedef uint32_t rows_4x4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t rows_4x2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t rows_2x2 __attribute__((ext_vector_type(2), aligned(2)));

// ONCE: past the caches.
template <bool ONCE, typename V> __device__ __forceinline__ V rows_get(const void *p)
{
    const V *q = reinterpret_cast<const V *>(p);
    if constexpr (ONCE)
        return __builtin_nontemporal_load(q);
    return *q;
}

// A piece as it lies in memory, requested now and used later.
template <typename TI, int E> struct RowPiece;
template <> struct RowPiece<float, 4> {
    u32x4 v;
    template <bool ONCE = false> __device__ __forceinline__ void load(const float *p) { v = rows_get<ONCE, rows_4x4>(p); }
    __device__ __forceinline__ float at(int e) const { return __uint_as_float(v[e]); }
};
template <> struct RowPiece<__bf16, 4> {
    uint2 v;
    template <bool ONCE = false> __device__ __forceinline__ void load(const __bf16 *p)
    {
        const rows_2x2 q = rows_get<ONCE, rows_2x2>(p);
        v = make_uint2(q[0], q[1]);
    }
    __device__ __forceinline__ float at(int e) const
    {
        const uint32_t w = e < 2 ? v.x : v.y;
        return __uint_as_float(e & 1 ? w & 0xFFFF0000u : w << 16);
    }
};
template <> struct RowPiece<__bf16, 8> {
    u32x4 v;
    template <bool ONCE = false> __device__ __forceinline__ void load(const __bf16 *p) { v = rows_get<ONCE, rows_4x2>(p); }
    __device__ __forceinline__ float at(int e) const { return chunk_elem<__bf16>(v, e); }
};
template <typename TI> struct RowPiece<TI, 1> {
    TI v;
    __device__ __forceinline__ void load(const TI *p) { v = *p; }
    __device__ __forceinline__ float at(int) const { return (float)v; }
};

__device__ __forceinline__ uint32_t rows_pack(float a, float b)
{
    const bf16x2 v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}

// Elements [from, E) of a piece to memory, rounded to nearest.
template <int E> __device__ __forceinline__ void rows_store(float *p, const float (&v)[E], int from)
{
    if constexpr (E == 4) {
        if (from == 0) {
            *reinterpret_cast<rows_4x4 *>(p) = rows_4x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                                        __float_as_uint(v[3])};
            return;
        }
    }
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (e >= from)
            p[e] = v[e];
}
template <int E> __device__ __forceinline__ void rows_store(__bf16 *p, const float (&v)[E], int from)
{
    if constexpr (E == 4) {
        if (from == 0) {
            *reinterpret_cast<rows_2x2 *>(p) = rows_2x2{rows_pack(v[0], v[1]), rows_pack(v[2], v[3])};
            return;
        }
    }
    if constexpr (E == 8) {
        if (from == 0) {
            *reinterpret_cast<rows_4x2 *>(p) = rows_4x2{rows_pack(v[0], v[1]), rows_pack(v[2], v[3]), rows_pack(v[4], v[5]),
                                                        rows_pack(v[6], v[7])};
            return;
        }
    }
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (e >= from)
            p[e] = (__bf16)v[e];
}

// Piece `i` of a row of d >= E columns: its first column, and the first of its
// elements that no other piece has (the last piece of a row whose width is no
// multiple of E begins inside the one before).
template <int E> __device__ __forceinline__ int rows_column(int i, int d, int &from)
{
    const int c = i * E, over = c + E - d;
    from = over > 0 ? over : 0;
    return c - from;
}

// The token id of a row as a 32-bit key: `V` where it is none of 0 .. V-1.
template <typename ID> __device__ __forceinline__ int token_key(const ID *ids, int64_t t, int V)
{
    const ID id = ids[t];
    return id >= 0 && id < (ID)V ? (int)id : V;
}

}  // namespace twell
