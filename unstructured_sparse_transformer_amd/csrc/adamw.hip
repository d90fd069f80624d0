// adamw.hip -- one AdamW step over many tensors (twell_adamw_step) and the
// values of 8-bit states (twell_adamw_unpack).
//
// Per element, with the bias corrections folded into two host constants:
//   g = grad * grad_scale
//   m = beta1 m + (1 - beta1) g          v = beta2 v + (1 - beta2) g^2
//   p = (1 - lr wd) p - size * m / (root * sqrt(v) + eps)
//   size = lr / (1 - beta1^step), root = 1 / sqrt(1 - beta2^step)
// all in fp32, every operation rounded by itself (no fused multiply-add), so
// that an 8-bit code never depends on how a compiler groups the sums.
//
// Bound by memory: p, m, v read and written, the gradient read, the 16-bit
// copy written, 30 bytes an element with 32-bit states and a bf16 gradient, 16
// with 8-bit states.  One launch covers up to AW_BATCH tensors: their table is
// in the kernel's arguments (no table to build in device memory, and a captured
// graph keeps it), a workgroup finds its tensor by a binary search over the
// first-workgroup numbers.  A thread holds 8 consecutive elements: 16-byte
// accesses throughout, and a block of 256 that shares a scale is 32 lanes, so
// its largest value needs no LDS.
//
// 8-bit states.  m: sign and 7 bits, sqrt(v): 8 bits, both the upper bits of
// the fp32 pattern of |x| / scale (3 and 4 bits of mantissa) with the exponent
// counted down from 1, i.e. 16 octaves of nearly constant relative steps; scale
// = the block's largest magnitude, fp32.  sqrt(v) instead of v halves the
// octaves that v's range takes.  Rounding is stochastic: beta2 near 1 changes v
// by less than half a step, which rounding to nearest would lose for ever; the
// noise is a hash of (seed, tensor, element), so a step is reproducible.  A
// root above 0 keeps at least the smallest code, since the update divides by it.
#include "adamw.h"
#include "twell_device.h"

namespace twell {

__device__ __forceinline__ uint32_t aw_noise(uint32_t key, int64_t i)
{
    uint32_t x = (uint32_t)i + (uint32_t)(i >> 32) * 0x5851F42Du + key;
    x = (x ^ (x >> 16)) * 0xA2C1B5D3u;
    x = (x ^ (x >> 15)) * 0x6D9E3C8Bu;
    return x ^ (x >> 16);
}

// Largest of `bits` (non-negative floats' patterns, NaN above all) over the
// 32 lanes of a half-wave.
__device__ __forceinline__ uint32_t half_wave_umax(uint32_t b)
{
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)b, m, 64);
        b = o > b ? o : b;
    }
    return b;
}

constexpr int AW_M_OFF = 889, AW_V_OFF = 1777;  // codes 127 and 255 are 1.0

__device__ __forceinline__ float aw_dec_m(uint32_t c, float scale)
{
    const uint32_t mag = c & 127u;
    const uint32_t b = mag ? (mag + AW_M_OFF) << 20 : 0u;
    return __uint_as_float(b | (mag ? (c & 128u) << 24 : 0u)) * scale;
}
__device__ __forceinline__ float aw_dec_r(uint32_t c, float scale)
{
    return __uint_as_float(c ? (c + AW_V_OFF) << 19 : 0u) * scale;
}

// Scale of a block whose largest magnitude has pattern `top`, and its
// reciprocal: a block below 1e-30 is held as zeros, one with an infinity or a
// NaN has scale NaN (every value of it reads back as NaN).
__device__ __forceinline__ void aw_scale(uint32_t top, float &scale, float &inv)
{
    const float t = __uint_as_float(top);
    scale = top >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : t < 1e-30f ? 0.f : t;
    inv = t < 1e-30f ? 0.f : 1.0f / t;
}

__device__ __forceinline__ uint32_t aw_code(float a, float inv, uint32_t noise, int shift, int off, int most)
{
    float q = a * inv;
    q = q < 1.f ? q : 1.f;
    int c = (int)((__float_as_uint(q) + noise) >> shift) - off;
    c = c < 0 ? 0 : c > most ? most : c;
    return (uint32_t)c;
}

__device__ __forceinline__ void load8f(const void *p, int64_t i, bool bf16, bool vec, int left, float (&o)[8])
{
    if (vec && left >= 8) {
        if (bf16) {
            const u32x4 c = ldg16((const __bf16 *)p + i);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                o[e] = chunk_elem<__bf16>(c, e);
        } else {
            const u32x4 a = ldg16((const float *)p + i), b = ldg16((const float *)p + i + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                o[e] = __uint_as_float(a[e]);
                o[e + 4] = __uint_as_float(b[e]);
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            o[e] = e >= left ? 0.f : bf16 ? (float)((const __bf16 *)p)[i + e] : ((const float *)p)[i + e];
    }
}

__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    const bf16x2 v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ void store8f(void *p, int64_t i, bool bf16, bool vec, int left, const float (&v)[8])
{
    if (vec && left >= 8) {
        if (bf16) {
            *reinterpret_cast<u32x4 *>((__bf16 *)p + i) =
                u32x4{pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7])};
        } else {
            float *q = (float *)p + i;
            *reinterpret_cast<float4 *>(q) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4 *>(q + 4) = make_float4(v[4], v[5], v[6], v[7]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < left) {
                if (bf16)
                    ((__bf16 *)p)[i + e] = (__bf16)v[e];
                else
                    ((float *)p)[i + e] = v[e];
            }
    }
}

__device__ __forceinline__ void load8c(const uint8_t *p, int64_t i, bool vec, int left, uint32_t (&c)[8])
{
    if (vec && left >= 8) {
        const uint2 w = *reinterpret_cast<const uint2 *>(p + i);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            c[e] = (w.x >> (8 * e)) & 255u;
            c[e + 4] = (w.y >> (8 * e)) & 255u;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            c[e] = e < left ? p[i + e] : 0u;
    }
}

__device__ __forceinline__ void store8c(uint8_t *p, int64_t i, bool vec, int left, const uint32_t (&c)[8])
{
    if (vec && left >= 8) {
        *reinterpret_cast<uint2 *>(p + i) = make_uint2(c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24,
                                                       c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < left)
                p[i + e] = (uint8_t)c[e];
    }
}

// The tensor whose workgroups include `wg`.
template <typename B> __device__ __forceinline__ int aw_find(const B &b, int wg)
{
    int lo = 0, hi = b.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (b.t[mid].chunk0 <= wg)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

template <bool CODED> __global__ __launch_bounds__(AW_THREADS) void adamw_kernel(AwBatch b)
{
#pragma clang fp contract(off)
    float gs = 1.f;
    if (b.grad_scale) {
        gs = *b.grad_scale;
        // a coefficient of 0, an infinity or a NaN: the gradients are not usable, nothing changes
        if (!(fabsf(gs) < __builtin_inff()) || gs == 0.f)
            return;
    }
    const AwTensor &t = b.t[aw_find(b, blockIdx.x)];
    const bool vec = t.flags & AW_VEC, pb = t.flags & AW_P_BF16, gb = t.flags & AW_G_BF16;
    const int64_t i0 = (int64_t)((int)blockIdx.x - t.chunk0) * AW_CHUNK + threadIdx.x * 8;
#pragma unroll 1
    for (int pass = 0; pass < AW_CHUNK / AW_PASS; ++pass) {
        const int64_t i = i0 + pass * AW_PASS;
        // whole blocks of 256 leave together: their 32 lanes share the largest value
        if ((i & ~(int64_t)(AW_QBLOCK - 1)) >= t.n)
            return;
        const int left = t.n - i >= 8 ? 8 : t.n - i > 0 ? (int)(t.n - i) : 0;
        float p[8], g[8], m[8], v[8];
        load8f(t.p, i, pb, vec, left, p);
        load8f(t.grad, i, gb, vec, left, g);
        if constexpr (CODED) {
            uint32_t cm[8], cv[8];
            load8c((const uint8_t *)t.m, i, vec, left, cm);
            load8c((const uint8_t *)t.v, i, vec, left, cv);
            const float sm = t.m_scale[i / AW_QBLOCK], sv = t.v_scale[i / AW_QBLOCK];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                m[e] = aw_dec_m(cm[e], sm);
                const float r = aw_dec_r(cv[e], sv);
                v[e] = r * r;
            }
        } else {
            load8f(t.m, i, false, vec, left, m);
            load8f(t.v, i, false, vec, left, v);
        }
        float r[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float ge = g[e] * gs;
            m[e] = m[e] * b.beta1 + ge * b.omb1;
            v[e] = v[e] * b.beta2 + (ge * ge) * b.omb2;
            r[e] = sqrtf(v[e]);
            p[e] = p[e] * t.decay - (m[e] / (r[e] * b.root + b.eps)) * b.size;
        }
        store8f(t.p, i, pb, vec, left, p);
        if (t.copy)
            store8f(t.copy, i, true, vec, left, p);
        if constexpr (CODED) {
            uint32_t am = 0, ar = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < left) {
                    const uint32_t bm = __float_as_uint(m[e]) & 0x7FFFFFFFu, br = __float_as_uint(r[e]) & 0x7FFFFFFFu;
                    am = bm > am ? bm : am;
                    ar = br > ar ? br : ar;
                }
            float sm, im, sr, ir;
            aw_scale(half_wave_umax(am), sm, im);
            aw_scale(half_wave_umax(ar), sr, ir);
            uint32_t cm[8], cv[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t x = aw_noise(t.key, i + e);
                cm[e] = aw_code(fabsf(m[e]), im, x & 0xFFFFFu, 20, AW_M_OFF, 127) | (m[e] < 0.f ? 128u : 0u);
                const uint32_t c = aw_code(r[e], ir, x >> 13, 19, AW_V_OFF, 255);
                cv[e] = c == 0 && r[e] * ir > 0.f ? 1u : c;
            }
            store8c((uint8_t *)t.m, i, vec, left, cm);
            store8c((uint8_t *)t.v, i, vec, left, cv);
            if ((threadIdx.x & 31) == 0) {
                t.m_scale[i / AW_QBLOCK] = sm;
                t.v_scale[i / AW_QBLOCK] = sr;
            }
        } else {
            store8f(t.m, i, false, vec, left, m);
            store8f(t.v, i, false, vec, left, v);
        }
    }
}

// m_values = m, v_values = sqrt(v)^2 of the codes: 2 + 8 bytes an element.
__global__ __launch_bounds__(AW_THREADS) void adamw_unpack_kernel(AwUnpack b)
{
    const auto &t = b.t[aw_find(b, blockIdx.x)];
    const int64_t i0 = (int64_t)((int)blockIdx.x - t.chunk0) * AW_CHUNK + threadIdx.x * 8;
#pragma unroll 1
    for (int pass = 0; pass < AW_CHUNK / AW_PASS; ++pass) {
        const int64_t i = i0 + pass * AW_PASS;
        if (i >= t.n)
            return;
        const int left = t.n - i >= 8 ? 8 : (int)(t.n - i);
        uint32_t cm[8], cv[8];
        load8c(t.m, i, t.vec, left, cm);
        load8c(t.v, i, t.vec, left, cv);
        const float sm = t.m_scale[i / AW_QBLOCK], sv = t.v_scale[i / AW_QBLOCK];
        float m[8], v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            m[e] = aw_dec_m(cm[e], sm);
            const float r = aw_dec_r(cv[e], sv);
            v[e] = r * r;
        }
        store8f(t.m_values, i, false, t.vec, left, m);
        store8f(t.v_values, i, false, t.vec, left, v);
    }
}

hipError_t launch_adamw(const AwBatch &b, bool coded, int chunks, hipStream_t s)
{
    if (coded)
        adamw_kernel<true><<<dim3(chunks), dim3(AW_THREADS), 0, s>>>(b);
    else
        adamw_kernel<false><<<dim3(chunks), dim3(AW_THREADS), 0, s>>>(b);
    return hipGetLastError();
}

hipError_t launch_adamw_unpack(const AwUnpack &b, int chunks, hipStream_t s)
{
    adamw_unpack_kernel<<<dim3(chunks), dim3(AW_THREADS), 0, s>>>(b);
    return hipGetLastError();
}

}  // namespace twell
