// act8.hip -- activations kept in 8 bits: packing and unpacking of rows
// (twell_act_pack, twell_act_unpack).
//
//   scale = max |x| / 127 over 32 consecutive elements of a row, in bf16, rounded up
//   code = round(x / scale) in 8 bits,  value = code * scale
// Linear codes: what a gradient needs of an activation is its absolute error (act
// and act' are smooth), which is at most half a step, 0.4% of the block's largest;
// a floating 8-bit code of 3 bits of mantissa is off by up to 6% of the value
// itself.  Bound by memory: 3.06 bytes an element of bf16 either way.
#include "act8.h"
#include "rows.h"

namespace twell {

typedef uint32_t a8_2x1 __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t a8_1x1 __attribute__((aligned(1)));

// Piece `piece` of E elements of row `row`; a row's pieces fill whole blocks.
template <int E> struct A8Place {
    int64_t row;
    int col, left;  // elements of the row from col on
    __device__ __forceinline__ A8Place(int64_t i, int pieces, int d)
    {
        row = i / pieces;
        col = (int)(i - row * pieces) * E;
        left = d - col;
    }
};

template <typename TI> __global__ __launch_bounds__(256) void act_pack_kernel(const TI *x, int T, int d, Packed8 to)
{
    constexpr int E = Elt<TI>::PER_CHUNK, LANES = A8_BLOCK / E;
    const int nb = (int)a8_blocks(d), pieces = nb * LANES;
    const int64_t n = (int64_t)T * pieces, step = (int64_t)gridDim.x * 256;
    for (int64_t i0 = (int64_t)blockIdx.x * 256; i0 < n; i0 += step) {
        const int64_t i = i0 + threadIdx.x;
        const bool on = i < n;
        const A8Place<E> at(on ? i : n - 1, pieces, d);
        const TI *q = x + at.row * d + at.col;
        float v[E];
        if (at.left >= E) {
            RowPiece<TI, E> r;
            r.load(q);
#pragma unroll
            for (int e = 0; e < E; ++e)
                v[e] = r.at(e);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e)
                v[e] = e < at.left ? (float)q[e] : 0.f;
        }
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e)
            top = a8_max(top, v[e]);
#pragma unroll
        for (int o = 1; o < LANES; o <<= 1)
            top = a8_max(top, __shfl_xor(top, o, 64));
        const A8Scale s(top);
        if (!on)
            continue;
        if (threadIdx.x % LANES == 0)
            to.scale[at.row * nb + at.col / A8_BLOCK] = s.bits;
        uint32_t c[E / 4];
#pragma unroll
        for (int k = 0; k < E / 4; ++k)
            c[k] = a8_codes(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3], s.inv);
        int8_t *o = to.code + at.row * d + at.col;
        if (at.left >= E) {
            if constexpr (E == 8)
                *reinterpret_cast<a8_2x1 *>(o) = a8_2x1{c[0], c[1]};
            else
                *reinterpret_cast<a8_1x1 *>(o) = c[0];
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (e < at.left)
                    o[e] = (int8_t)(c[e / 4] >> (8 * (e % 4)));
        }
    }
}

template <typename TO> __global__ __launch_bounds__(256) void act_unpack_kernel(Packed8 from, int T, int d, TO *out)
{
    constexpr int E = Elt<TO>::PER_CHUNK;
    const int nb = (int)a8_blocks(d), pieces = (d + E - 1) / E;
    const int64_t n = (int64_t)T * pieces, step = (int64_t)gridDim.x * 256;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += step) {
        const A8Place<E> at(i, pieces, d);
        const int8_t *q = from.code + at.row * d + at.col;
        const float s = a8_scale(from.scale[at.row * nb + at.col / A8_BLOCK]);
        TO *o = out + at.row * d + at.col;
        if (at.left >= E) {
            uint32_t c[E / 4];
            if constexpr (E == 8) {
                const a8_2x1 w = *reinterpret_cast<const a8_2x1 *>(q);
                c[0] = w[0];
                c[1] = w[1];
            } else {
                c[0] = *reinterpret_cast<const a8_1x1 *>(q);
            }
            float v[E];
#pragma unroll
            for (int e = 0; e < E; ++e)
                v[e] = a8_value(c[e / 4], e % 4, s);
            rows_store<E>(o, v, 0);
        } else {
            for (int e = 0; e < at.left; ++e)
                o[e] = (TO)((float)q[e] * s);
        }
    }
}

// ------------------------------------------------------------------ host
static dim3 a8_grid(int64_t threads)
{
    const int64_t wgs = (threads + 255) / 256;
    return dim3((unsigned)(wgs < 16384 ? wgs : 16384));
}

hipError_t launch_act_pack(int vdtype, const void *x, int T, int d, Packed8 to, hipStream_t s)
{
    const int64_t blocks = (int64_t)T * a8_blocks(d);
    if (vdtype == 1)
        act_pack_kernel<__bf16><<<a8_grid(blocks * 4), dim3(256), 0, s>>>((const __bf16 *)x, T, d, to);
    else
        act_pack_kernel<float><<<a8_grid(blocks * 8), dim3(256), 0, s>>>((const float *)x, T, d, to);
    return hipGetLastError();
}

hipError_t launch_act_unpack(int vdtype, Packed8 from, int T, int d, void *out, hipStream_t s)
{
    if (vdtype == 1)
        act_unpack_kernel<__bf16><<<a8_grid((int64_t)T * ((d + 7) / 8)), dim3(256), 0, s>>>(from, T, d, (__bf16 *)out);
    else
        act_unpack_kernel<float><<<a8_grid((int64_t)T * ((d + 3) / 4)), dim3(256), 0, s>>>(from, T, d, (float *)out);
    return hipGetLastError();
}

}  // namespace twell
