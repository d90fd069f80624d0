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
struct A8Scale {
    uint16_t bits;
    float inv;
    __device__ __forceinline__ A8Scale(float top)
    {
        const uint32_t b = (__float_as_uint(top / 127.f) + 0xFFFFu) >> 16;
        const bool fine = top < INFINITY;
        bits = fine ? top < 1e-30f ? 0 : (uint16_t)b : 0x7FC0;
        inv = fine && !(top < 1e-30f) ? 1.f / __uint_as_float(b << 16) : 0.f;
    }
};

// The codes of 4 values, one a byte: round to nearest even, by an addition whose
// result has the whole number in its lowest bits (after the product's own
// rounding: a code does not depend on whether a compiler fuses the two).
__device__ __forceinline__ uint32_t a8_codes(float a, float b, float c, float d, float inv)
{
#pragma clang fp contract(off)
    constexpr float WHOLE = 12582912.f;  // 1.5 2^23
    const uint32_t x = __float_as_uint(a * inv + WHOLE), y = __float_as_uint(b * inv + WHOLE),
                   z = __float_as_uint(c * inv + WHOLE), w = __float_as_uint(d * inv + WHOLE);
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
