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
// copy written, 28 bytes an element with 32-bit states and a bf16 gradient, 16
// with 8-bit states.  One launch covers up to AW_BATCH tensors: their table is
// in the kernel's arguments (no table to build in device memory, and a captured
// graph keeps it), a workgroup finds its tensor by a binary search over the
// first-workgroup numbers.  A lane holds 4 consecutive elements of each of two
// blocks of 256: a wave's fp32 accesses are 16 bytes a lane without gaps (8
// consecutive elements a lane left gaps of 16 bytes between a store's pieces),
// and the 256 elements that share a scale are one wave, so their largest value
// needs no LDS.  All but the copies is read and written past the caches
// (nontemporal): nothing of it is used again before the next step.  Measured: 235
// us for 50 M elements with 32-bit states (6.0 TB/s; 268 us through the caches),
// 311 us for 100 M with 8-bit states (5.2 TB/s; 326 us), 176 us to unpack those
// (5.7 TB/s; 184 us).
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

#include <type_traits>

namespace twell {
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint32_t aw_noise(uint32_t key, int64_t i)
{
    uint32_t x = (uint32_t)i + (uint32_t)(i >> 32) * 0x5851F42Du + key;
    x = (x ^ (x >> 16)) * 0xA2C1B5D3u;
    x = (x ^ (x >> 15)) * 0x6D9E3C8Bu;
    return x ^ (x >> 16);
}

// Largest of `b` (non-negative floats' patterns, NaN above all) over the wave,
// with DPP row shifts and row broadcasts; lanes without a source count as 0.
__device__ __forceinline__ uint32_t wave_umax(uint32_t b)
{
    auto step = [&](auto ctrl, auto rows) {
        const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)b, decltype(ctrl)::value, decltype(rows)::value,
                                                                 0xf, false);
        b = o > b ? o : b;
    };
    using std::integral_constant;
    step(integral_constant<int, 0x111>{}, integral_constant<int, 0xf>{});  // row_shr:1
    step(integral_constant<int, 0x112>{}, integral_constant<int, 0xf>{});  // row_shr:2
    step(integral_constant<int, 0x114>{}, integral_constant<int, 0xf>{});  // row_shr:4
    step(integral_constant<int, 0x118>{}, integral_constant<int, 0xf>{});  // row_shr:8
    step(integral_constant<int, 0x142>{}, integral_constant<int, 0xa>{});  // row_bcast:15
    step(integral_constant<int, 0x143>{}, integral_constant<int, 0xc>{});  // row_bcast:31
    return (uint32_t)__builtin_amdgcn_readlane((int)b, 63);
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

// 4 elements from index i, `left` of them inside the tensor; WIDE: all 4, and
// aligned for one access.  The types are the template's: a conversion under a
// run-time branch would wait for its load there, one load after another.
template <bool BF16, bool WIDE> __device__ __forceinline__ void load4f(const void *p, int64_t i, int left, float (&o)[4])
{
    if constexpr (WIDE) {
        if constexpr (BF16) {
            const u32x2 c = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>((const __bf16 *)p + i));
            o[0] = __uint_as_float(c.x << 16);
            o[1] = __uint_as_float(c.x & 0xFFFF0000u);
            o[2] = __uint_as_float(c.y << 16);
            o[3] = __uint_as_float(c.y & 0xFFFF0000u);
        } else {
            const f32x4 c = __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>((const float *)p + i));
            o[0] = c.x;
            o[1] = c.y;
            o[2] = c.z;
            o[3] = c.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            o[e] = e >= left ? 0.f : BF16 ? (float)((const __bf16 *)p)[i + e] : ((const float *)p)[i + e];
    }
}

__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    const bf16x2 v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}

// KEEP: read soon (the layers' copies); the rest leaves the caches at once.
template <bool BF16, bool WIDE, bool KEEP = false>
__device__ __forceinline__ void store4f(void *p, int64_t i, int left, const float (&v)[4])
{
    if constexpr (WIDE) {
        if constexpr (BF16 && KEEP)
            *reinterpret_cast<u32x2 *>((__bf16 *)p + i) = u32x2{pack2(v[0], v[1]), pack2(v[2], v[3])};
        else if constexpr (BF16)
            __builtin_nontemporal_store(u32x2{pack2(v[0], v[1]), pack2(v[2], v[3])},
                                        reinterpret_cast<u32x2 *>((__bf16 *)p + i));
        else
            __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, reinterpret_cast<f32x4 *>((float *)p + i));
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < left) {
                if constexpr (BF16)
                    ((__bf16 *)p)[i + e] = (__bf16)v[e];
                else
                    ((float *)p)[i + e] = v[e];
            }
    }
}

template <bool WIDE> __device__ __forceinline__ uint32_t load4c(const uint8_t *p, int64_t i, int left)
{
    if constexpr (WIDE)
        return __builtin_nontemporal_load(reinterpret_cast<const uint32_t *>(p + i));
    uint32_t c = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e < left)
            c |= (uint32_t)p[i + e] << (8 * e);
    return c;
}

template <bool WIDE> __device__ __forceinline__ void store4c(uint8_t *p, int64_t i, int left, uint32_t c)
{
    if constexpr (WIDE) {
        __builtin_nontemporal_store(c, reinterpret_cast<uint32_t *>(p + i));
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < left)
                p[i + e] = (uint8_t)(c >> (8 * e));
    }
}

__device__ __forceinline__ int aw_left(int64_t n, int64_t i) { return n - i >= 4 ? 4 : n - i > 0 ? (int)(n - i) : 0; }

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

// The step on one workgroup's elements, from c0 on.
template <bool CODED, bool PB, bool GB, bool WIDE>
__device__ __forceinline__ void adamw_chunk(const AwBatch &b, const AwTensor &t, int64_t c0, float gs)
{
#pragma clang fp contract(off)
    const int lane = threadIdx.x & 63;
    const int64_t w0 = c0 + (threadIdx.x >> 6) * (2 * AW_QBLOCK);
#pragma unroll 1
    for (int pass = 0; pass < b.passes; ++pass) {
        const int64_t b0 = w0 + pass * AW_PASS;  // the wave's first block
        if (!WIDE && b0 >= t.n)
            return;
        float p[2][4], g[2][4], m[2][4], v[2][4];
        uint32_t cm[2], cv[2];
        float sm[2], sv[2];
        int left[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t i = b0 + h * AW_QBLOCK + lane * 4;
            left[h] = WIDE ? 4 : aw_left(t.n, i);
            load4f<PB, WIDE>(t.p, i, left[h], p[h]);
            load4f<GB, WIDE>(t.grad, i, left[h], g[h]);
            if constexpr (CODED) {
                cm[h] = load4c<WIDE>((const uint8_t *)t.m, i, left[h]);
                cv[h] = load4c<WIDE>((const uint8_t *)t.v, i, left[h]);
                const int64_t q = (WIDE || b0 + h * AW_QBLOCK < t.n ? b0 + h * AW_QBLOCK : b0) / AW_QBLOCK;
                sm[h] = t.m_scale[q];
                sv[h] = t.v_scale[q];
            } else {
                load4f<false, WIDE>(t.m, i, left[h], m[h]);
                load4f<false, WIDE>(t.v, i, left[h], v[h]);
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t i = b0 + h * AW_QBLOCK + lane * 4;
            float r[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (CODED) {
                    m[h][e] = aw_dec_m((cm[h] >> (8 * e)) & 255u, sm[h]);
                    const float root = aw_dec_r((cv[h] >> (8 * e)) & 255u, sv[h]);
                    v[h][e] = root * root;
                }
                const float ge = g[h][e] * gs;
                m[h][e] = m[h][e] * b.beta1 + ge * b.omb1;
                v[h][e] = v[h][e] * b.beta2 + (ge * ge) * b.omb2;
                r[e] = sqrtf(v[h][e]);
                p[h][e] = p[h][e] * t.decay - (m[h][e] / (r[e] * b.root + b.eps)) * b.size;
            }
            store4f<PB, WIDE>(t.p, i, left[h], p[h]);
            if (t.copy)
                store4f<true, WIDE, true>(t.copy, i, left[h], p[h]);
            if constexpr (CODED) {
                if (!WIDE && b0 + h * AW_QBLOCK >= t.n)
                    return;
                uint32_t am = 0, ar = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (e < left[h]) {
                        const uint32_t bm = __float_as_uint(m[h][e]) & 0x7FFFFFFFu;
                        const uint32_t br = __float_as_uint(r[e]) & 0x7FFFFFFFu;
                        am = bm > am ? bm : am;
                        ar = br > ar ? br : ar;
                    }
                float im, ir;
                aw_scale(wave_umax(am), sm[h], im);
                aw_scale(wave_umax(ar), sv[h], ir);
                uint32_t om = 0, ov = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t x = aw_noise(t.key, i + e);
                    om |= (aw_code(fabsf(m[h][e]), im, x & 0xFFFFFu, 20, AW_M_OFF, 127) | (m[h][e] < 0.f ? 128u : 0u))
                          << (8 * e);
                    const uint32_t c = aw_code(r[e], ir, x >> 13, 19, AW_V_OFF, 255);
                    ov |= (c == 0 && r[e] * ir > 0.f ? 1u : c) << (8 * e);
                }
                store4c<WIDE>((uint8_t *)t.m, i, left[h], om);
                store4c<WIDE>((uint8_t *)t.v, i, left[h], ov);
                if (lane == 0) {
                    t.m_scale[b0 / AW_QBLOCK + h] = sm[h];
                    t.v_scale[b0 / AW_QBLOCK + h] = sv[h];
                }
            } else {
                store4f<false, WIDE>(t.m, i, left[h], m[h]);
                store4f<false, WIDE>(t.v, i, left[h], v[h]);
            }
        }
    }
}

template <bool CODED> __global__ __launch_bounds__(AW_THREADS) void adamw_kernel(AwBatch b)
{
    float gs = 1.f;
    if (b.grad_scale) {
        gs = *b.grad_scale;
        // a coefficient of 0, an infinity or a NaN: the gradients are not usable, nothing changes
        if (!(fabsf(gs) < __builtin_inff()) || gs == 0.f)
            return;
    }
    const AwTensor &t = b.t[aw_find(b, blockIdx.x)];
    const int chunk = b.passes * AW_PASS;
    const int64_t c0 = (int64_t)((int)blockIdx.x - t.chunk0) * chunk;
    const bool pb = t.flags & AW_P_BF16, gb = t.flags & AW_G_BF16;
    if ((t.flags & AW_VEC) && c0 + chunk <= t.n) {
        if (pb)
            gb ? adamw_chunk<CODED, true, true, true>(b, t, c0, gs) : adamw_chunk<CODED, true, false, true>(b, t, c0, gs);
        else
            gb ? adamw_chunk<CODED, false, true, true>(b, t, c0, gs) : adamw_chunk<CODED, false, false, true>(b, t, c0, gs);
    } else {
        if (pb)
            gb ? adamw_chunk<CODED, true, true, false>(b, t, c0, gs) : adamw_chunk<CODED, true, false, false>(b, t, c0, gs);
        else
            gb ? adamw_chunk<CODED, false, true, false>(b, t, c0, gs) : adamw_chunk<CODED, false, false, false>(b, t, c0, gs);
    }
}

// m_values = m, v_values = sqrt(v)^2 of the codes: 2 + 8 bytes an element.
template <typename T, int PASSES, bool WIDE> __device__ __forceinline__ void unpack_chunk(T t, int64_t c0)
{
    constexpr int N = PASSES * AW_PASS / AW_THREADS / 4;
    uint32_t cm[N], cv[N];
    float sm[N], sv[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int64_t i = c0 + k * (AW_THREADS * 4) + threadIdx.x * 4;
        const int left = WIDE ? 4 : aw_left(t.n, i);
        cm[k] = load4c<WIDE>(t.m, i, left);
        cv[k] = load4c<WIDE>(t.v, i, left);
        sm[k] = left ? t.m_scale[i / AW_QBLOCK] : 0.f;
        sv[k] = left ? t.v_scale[i / AW_QBLOCK] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int64_t i = c0 + k * (AW_THREADS * 4) + threadIdx.x * 4;
        const int left = WIDE ? 4 : aw_left(t.n, i);
        float m[4], v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            m[e] = aw_dec_m((cm[k] >> (8 * e)) & 255u, sm[k]);
            const float r = aw_dec_r((cv[k] >> (8 * e)) & 255u, sv[k]);
            v[e] = r * r;
        }
        store4f<false, WIDE>(t.m_values, i, left, m);
        store4f<false, WIDE>(t.v_values, i, left, v);
    }
}

template <int PASSES> __global__ __launch_bounds__(AW_THREADS) void adamw_unpack_kernel(AwUnpack b)
{
    const auto &t = b.t[aw_find(b, blockIdx.x)];
    const int64_t c0 = (int64_t)((int)blockIdx.x - t.chunk0) * (PASSES * AW_PASS);
    if (t.vec && c0 + PASSES * AW_PASS <= t.n)
        unpack_chunk<decltype(t), PASSES, true>(t, c0);
    else
        unpack_chunk<decltype(t), PASSES, false>(t, c0);
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
    if (b.passes == AW_PASSES)
        adamw_unpack_kernel<AW_PASSES><<<dim3(chunks), dim3(AW_THREADS), 0, s>>>(b);
    else
        adamw_unpack_kernel<1><<<dim3(chunks), dim3(AW_THREADS), 0, s>>>(b);
    return hipGetLastError();
}

}  // namespace twell
