// act8.h -- activations kept in 8 bits (host and device side).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace twell {

constexpr int A8_BLOCK = 32;  // consecutive elements of a row that share a scale

__host__ __device__ inline int64_t a8_blocks(int64_t d) { return (d + A8_BLOCK - 1) / A8_BLOCK; }

// Rows of d: code [T][d], scale [T][a8_blocks(d)] in bf16.
struct Packed8 {
    int8_t *code;
    uint16_t *scale;
};

hipError_t launch_act_pack(int vdtype, const void *x, int T, int d, Packed8 to, hipStream_t s);
hipError_t launch_act_unpack(int vdtype, Packed8 from, int T, int d, void *out, hipStream_t s);

#ifdef __HIPCC__
// The larger magnitude of what has been seen and x, or NaN if either is.
__device__ __forceinline__ float a8_max(float a, float x) { return __builtin_elementwise_maximum(a, __builtin_fabsf(x)); }

// A block's scale from its largest magnitude: 127 steps reach it.  The step is
// held in bf16, rounded up, so that no code passes 127.  A block below 1e-30 is
// held as zeros; one with an infinity or a NaN has scale NaN and reads back as NaN
// as a whole.
//
// Both quotients are those of a correctly rounded division, in a third of its
// operations (of the gated product's largest tile a lane makes 8 scales): an estimate and
// one exact remainder.  A quotient by 127, or of 1 by a step of 8 bits of mantissa,
// is at least 1 / 512 of a unit in the last place away from where rounding turns, and
// the corrected estimate within 2^-20 of one.
struct A8Scale {
    uint16_t bits;
    float inv;
    __device__ __forceinline__ A8Scale(float top)
    {
        constexpr float R127 = 1.f / 127.f;
        const float q = top * R127;
        const uint32_t b = (__float_as_uint(fmaf(fmaf(-q, 127.f, top), R127, q)) + 0xFFFFu) & 0xFFFF0000u;
        const float step = __uint_as_float(b), r = __builtin_amdgcn_rcpf(step);
        const bool fine = top < INFINITY, some = fine && !(top < 1e-30f);
        bits = some ? (uint16_t)(b >> 16) : fine ? 0 : 0x7FC0;
        inv = some ? fmaf(fmaf(-step, r, 1.f), r, r) : 0.f;
    }
};

// How a value becomes a code: the product with 1 / step rounded by itself first, so
// that a code does not depend on whether a compiler fuses the two; in one operation
// (values that no other operation has in these 32 bits); or so, and values above 0 at
// least 1.
enum A8Round { A8_TWICE, A8_FUSED, A8_SIGN };

// A value's code in the lowest byte: round to nearest even, by an addition whose
// result has the whole number in its lowest bits.
template <A8Round R> __device__ __forceinline__ uint32_t a8_whole(float v, float inv)
{
#pragma clang fp contract(off)
    constexpr float WHOLE = 12582912.f;  // 1.5 2^23
    const float w = R == A8_TWICE ? v * inv + WHOLE : __builtin_fmaf(v, inv, WHOLE);
    const float up = R == A8_SIGN && v > 0.f ? WHOLE + 1.f : w;
    return __float_as_uint(w > up ? w : up);
}

// The codes of 4 values, one a byte.
template <A8Round R = A8_TWICE> __device__ __forceinline__ uint32_t a8_codes(float a, float b, float c, float d, float inv)
{
    const uint32_t x = a8_whole<R>(a, inv), y = a8_whole<R>(b, inv), z = a8_whole<R>(c, inv), w = a8_whole<R>(d, inv);
    return __builtin_amdgcn_perm(__builtin_amdgcn_perm(w, z, 0x0C0C0400u), __builtin_amdgcn_perm(y, x, 0x0C0C0400u), 0x05040100u);
}

// The value of code `e` (0 .. 3) of four.
__device__ __forceinline__ float a8_value(uint32_t codes, int e, float scale)
{
    return (float)(int8_t)(codes >> (8 * e)) * scale;
}
__device__ __forceinline__ float a8_scale(uint16_t bits) { return __uint_as_float((uint32_t)bits << 16); }
#endif

}  // namespace twell
