// act8.hip -- activations kept in 8 bits: packing and unpacking of rows
// (twell_act_pack, twell_act_unpack).
//
//   scale = max |x| / 127 over 32 consecutive elements of a row, in bf16, rounded up
//   code = round(x / scale) in 8 bits,  value = code * scale
// Linear codes: what a gradient needs of an activation is its absolute error (act
// and act' are smooth; ReLU's slope needs its sign, see glu.hip), which is at most
// half a step, 0.4% of the block's largest;
// a floating 8-bit code of 3 bits of mantissa is off by up to 6% of the value
// itself.  Bound by memory: 3.06 bytes an element of bf16 either way
// (8192 x 8192: packed in 35.5 us, 5.8 TB/s; unpacked, from caches in part, in 30 us).
#include "act8.h"
#include "rows.h"

namespace twell {

typedef uint32_t a8_2x1 __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t a8_1x1 __attribute__((aligned(1)));

// Item first + add of all rows' pieces of E elements.  A workgroup's first row is
// found once, in 64 bits; its threads count on from there.
template <int E> struct A8Place {
    int64_t row;
    int col, left;  // elements of the row from col on
    __device__ __forceinline__ A8Place(int64_t first, uint32_t add, int pieces, int d)
    {
        const int64_t r0 = first / pieces;
        const uint32_t r = (uint32_t)(first - r0 * pieces) + add, up = r / (uint32_t)pieces;
        row = r0 + up;
        col = (int)(r - up * (uint32_t)pieces) * E;
        left = d - col;
    }
};

// U: items of a thread, requested together; ONCE: read past the caches.
template <typename TI, int A8_U, bool ONCE> __global__ __launch_bounds__(256) void act_pack_kernel(const TI *x, int T, int d, Packed8 to)
{
    constexpr int E = Elt<TI>::PER_CHUNK, LANES = A8_BLOCK / E;
    const int nb = (int)a8_blocks(d), pieces = nb * LANES;
    const int64_t first = (int64_t)blockIdx.x * (256 * A8_U);
    RowPiece<TI, E> r[A8_U];
#pragma unroll
    for (int u = 0; u < A8_U; ++u) {
        const A8Place<E> at(first, u * 256 + threadIdx.x, pieces, d);
        if (at.row < T && at.left >= E)
            r[u].template load<ONCE>(x + at.row * d + at.col);
    }
#pragma unroll
    for (int u = 0; u < A8_U; ++u) {
        const A8Place<E> at(first, u * 256 + threadIdx.x, pieces, d);
        const bool on = at.row < T;
        float v[E];
#pragma unroll
        for (int e = 0; e < E; ++e)
            v[e] = r[u].at(e);
        if (!on || at.left < E) {
#pragma unroll
            for (int e = 0; e < E; ++e)
                v[e] = on && e < at.left ? (float)x[at.row * d + at.col + e] : 0.f;
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

template <typename TO, int A8_U> __global__ __launch_bounds__(256) void act_unpack_kernel(Packed8 from, int T, int d, TO *out)
{
    constexpr int E = Elt<TO>::PER_CHUNK;
    const int nb = (int)a8_blocks(d), pieces = (d + E - 1) / E;
    const int64_t first = (int64_t)blockIdx.x * (256 * A8_U);
    uint32_t c[A8_U][E / 4];
    uint16_t s[A8_U];
#pragma unroll
    for (int u = 0; u < A8_U; ++u) {
        const A8Place<E> at(first, u * 256 + threadIdx.x, pieces, d);
        if (at.row >= T)
            continue;
        s[u] = from.scale[at.row * nb + at.col / A8_BLOCK];
        const int8_t *q = from.code + at.row * d + at.col;
        if (at.left < E)
            continue;
        if constexpr (E == 8) {
            const a8_2x1 w = *reinterpret_cast<const a8_2x1 *>(q);
            c[u][0] = w[0];
            c[u][1] = w[1];
        } else {
            c[u][0] = *reinterpret_cast<const a8_1x1 *>(q);
        }
    }
#pragma unroll
    for (int u = 0; u < A8_U; ++u) {
        const A8Place<E> at(first, u * 256 + threadIdx.x, pieces, d);
        if (at.row >= T)
            continue;
        TO *o = out + at.row * d + at.col;
        const float scale = a8_scale(s[u]);
        if (at.left >= E) {
            float v[E];
#pragma unroll
            for (int e = 0; e < E; ++e)
                v[e] = a8_value(c[u][e / 4], e % 4, scale);
            rows_store<E>(o, v, 0);
        } else {
            for (int e = 0; e < at.left; ++e)
                o[e] = (TO)((float)from.code[at.row * d + at.col + e] * scale);
        }
    }
}

// ------------------------------------------------------------------ host
// From A8_LARGE elements on (more than the L2s hold) two items a thread, past the
// caches: calls of 8192 x 8192 fp32 59.7 and 64.1 us, 63.5 and 70.1 with one through
// them; bf16 35.2 and 30.3, with one 34.7 and 31.6; the kernels of 64 x 1001 fp32 3.8 us
// with two, 2.8 with one.
constexpr int64_t A8_LARGE = (int64_t)1 << 24;

static dim3 a8_grid(int64_t items, int each) { return dim3((unsigned)((items + 256 * each - 1) / (256 * each))); }

template <typename TI> static hipError_t run_pack(const void *x, int T, int d, Packed8 to, hipStream_t s)
{
    const int64_t items = (int64_t)T * a8_blocks(d) * (A8_BLOCK / Elt<TI>::PER_CHUNK);
    if ((int64_t)T * d >= A8_LARGE)
        act_pack_kernel<TI, 2, true><<<a8_grid(items, 2), dim3(256), 0, s>>>((const TI *)x, T, d, to);
    else
        act_pack_kernel<TI, 1, false><<<a8_grid(items, 1), dim3(256), 0, s>>>((const TI *)x, T, d, to);
    return hipGetLastError();
}

template <typename TO> static hipError_t run_unpack(Packed8 from, int T, int d, void *out, hipStream_t s)
{
    constexpr int E = Elt<TO>::PER_CHUNK;
    const int64_t items = (int64_t)T * ((d + E - 1) / E);
    if ((int64_t)T * d >= A8_LARGE)
        act_unpack_kernel<TO, 2><<<a8_grid(items, 2), dim3(256), 0, s>>>(from, T, d, (TO *)out);
    else
        act_unpack_kernel<TO, 1><<<a8_grid(items, 1), dim3(256), 0, s>>>(from, T, d, (TO *)out);
    return hipGetLastError();
}

hipError_t launch_act_pack(int vdtype, const void *x, int T, int d, Packed8 to, hipStream_t s)
{
    return vdtype == 1 ? run_pack<__bf16>(x, T, d, to, s) : run_pack<float>(x, T, d, to, s);
}

hipError_t launch_act_unpack(int vdtype, Packed8 from, int T, int d, void *out, hipStream_t s)
{
    return vdtype == 1 ? run_unpack<__bf16>(from, T, d, out, s) : run_unpack<float>(from, T, d, out, s);
}

}  // namespace twell
