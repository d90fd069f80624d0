// block_norm.hip -- the norms before and after a block, fused with the
// block's gate, residual scale and residual sum (twell_block_norm_forward,
// twell_block_norm_backward).
//
//   p = norm(y; w_post, b_post)            (or y)
//   r = res + alpha * gate * p,  out = r   (or r = res)
//   n = norm(r; w_pre, b_pre)
// norm(v) = (v - mean) * rstd * w + b with mean = 0 for the RMS kind and
// rstd = 1 / sqrt(mean((v - mean)^2) + eps).
//
// Backward, with vhat = (v - mean) rstd and g = dnorm * w:
//   dv = rstd (g - vhat mean(g vhat) [- mean(g)]),
//   dr = dout + dv_pre, dres = dr, dgate = sum alpha p dr, dy = dv_post of alpha gate dr,
//   dw = sum over rows of dnorm vhat, db = sum over rows of dnorm.
// The statistics come again from the rows that the backward pass reads anyway.
//
// Bound by memory: every row of every tensor moves once.  A row is held in
// registers by NT threads of 8 elements (NT = 2 to 1024 by the width), so a
// mean and a variance are two passes over registers, not over memory.  All
// sums are fp32: per thread, then over the row's lanes by DPP, then over the
// waves through LDS.  8192 x 2048: forward 26 us in bf16 (134 MB, 5.2 TB/s),
// backward 53 us in bf16 (201 MB) and 88 us with fp32 streams (403 MB, 4.6 TB/s),
// 6 us of them the second launch's sums of the partial rows; 29 and 97 us (forward,
// and backward in fp32) where a call's inputs are others than the last one's.
#include "block_norm.h"
#include "twell_device.h"
#include "wave_ops.h"

#include <type_traits>

namespace twell {

// How a row's columns lie on its NT threads, 8 a thread: BN_8 eight consecutive
// ones (16 bytes of bf16); BN_4
// two groups of four, the second 4 NT columns on (16 bytes of fp32, so that a
// wave's accesses to fp32 have no gaps); BN_END, for any width from 8 on and any
// alignment of the elements, as BN_8, but counted from the row's end: the first
// thread's eight columns overlap with the second's, which get the same values from
// both and count once in sums (both lie in one wave, which has loaded them before
// it stores: a result may take its input's place); BN_ANY, for widths below 8, one by one.  (One by one at any
// odd width: 8192 x 1001 forward in bf16 22.5 us, 16.8 so, backward 52 and 39.)
enum BnLay { BN_ANY, BN_8, BN_4, BN_END };

// Whether element e of a thread is one of the row's columns.
template <BnLay L, int NT> __device__ __forceinline__ bool bn_in(int tid, int e, int d)
{
    return (L == BN_END   ? tid * 8
            : L == BN_8   ? tid * 8 + e
            : L == BN_4   ? (e >> 2) * 4 * NT + tid * 4 + (e & 3)
                          : e * NT + tid) < d;
}

// BN_END: the first column of a thread.
__device__ __forceinline__ int bn_end(int tid, int d)
{
    const int c = tid * 8 - (-d & 7);
    return c > 0 ? c : 0;
}

// v where element e counts in the row's sums (elements past d are 0).
template <BnLay L> __device__ __forceinline__ float bn_once(float v, int tid, int e, int d)
{
    return L == BN_END && tid == 0 && e >= 8 - (-d & 7) ? 0.f : v;
}

typedef uint32_t u32x4_al2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_al4 __attribute__((ext_vector_type(4), aligned(4)));

// Keeps the compiler from holding an address per element and tensor over a loop
// of rows (more than 256 registers): they are one addition each.
__device__ __forceinline__ void bn_forget(int &v) { asm volatile("" : "+v"(v)); }

// 8 elements of a row as they lie in memory, requested now and used later.
struct Raw8 {
    u32x4 a, b;
};

template <bool ONCE, typename V = u32x4> __device__ __forceinline__ u32x4 bn_ld16(const void *p)
{
    const V *q = reinterpret_cast<const V *>(p);
    if constexpr (ONCE)
        return __builtin_nontemporal_load(q);
    return *q;
}

template <BnLay L, int NT, bool ONCE = false>
__device__ __forceinline__ Raw8 bn_load(BnTensor t, int64_t row, int d, int tid)
{
    Raw8 r{};
    if constexpr (L == BN_8) {
        if (tid * 8 < d) {
            if (t.bf16) {
                r.a = bn_ld16<ONCE>((const __bf16 *)t.p + row * d + (uint32_t)(tid * 8));
            } else {
                const float *q = (const float *)t.p + row * d + (uint32_t)(tid * 8);
                r.a = bn_ld16<ONCE>(q);
                r.b = bn_ld16<ONCE>(q + 4);
            }
        }
    } else if constexpr (L == BN_END) {
        if (tid * 8 < d) {
            // (through the caches: threads share lines)
            const uint32_t c = bn_end(tid, d);
            if (t.bf16) {
                r.a = bn_ld16<false, u32x4_al2>((const __bf16 *)t.p + row * d + c);
            } else {
                const float *q = (const float *)t.p + row * d + c;
                r.a = bn_ld16<false, u32x4_al4>(q);
                r.b = bn_ld16<false, u32x4_al4>(q + 4);
            }
        }
    } else if constexpr (L == BN_4) {
        const int c0 = tid * 4, c1 = 4 * NT + tid * 4;
        if (t.bf16) {
            const __bf16 *q = (const __bf16 *)t.p + row * d;
            uint2 x{}, y{};
            if (c0 < d)
                x = *reinterpret_cast<const uint2 *>(q + c0);
            if (c1 < d)
                y = *reinterpret_cast<const uint2 *>(q + c1);
            r.a = u32x4{x.x, x.y, y.x, y.y};
        } else {
            const float *q = (const float *)t.p + row * d;
            if (c0 < d)
                r.a = bn_ld16<ONCE>(q + c0);
            if (c1 < d)
                r.b = bn_ld16<ONCE>(q + c1);
        }
    } else {
        // columns past d read column d - 1 and count as 0: no load waits behind a branch
        uint32_t w[8];
        bn_forget(tid);
        if (t.bf16) {
            const uint16_t *q = (const uint16_t *)t.p + row * d;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                w[e] = q[(uint32_t)(e * NT + tid < d ? e * NT + tid : d - 1)];
        } else {
            const uint32_t *q = (const uint32_t *)t.p + row * d;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                w[e] = q[(uint32_t)(e * NT + tid < d ? e * NT + tid : d - 1)];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            w[e] = e * NT + tid < d ? w[e] : 0u;
        r.a = t.bf16 ? u32x4{w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16}
                     : u32x4{w[0], w[1], w[2], w[3]};
        r.b = u32x4{w[4], w[5], w[6], w[7]};
    }
    return r;
}

__device__ __forceinline__ void bn_values(const Raw8 &r, int bf16, float (&v)[8])
{
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float h = chunk_elem<__bf16>(r.a, e);
        const float f = __uint_as_float(e < 4 ? r.a[e & 3] : r.b[e & 3]);
        v[e] = bf16 ? h : f;
    }
}

__device__ __forceinline__ uint32_t bn_pack(float a, float b)
{
    const bf16x2 v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}

template <BnLay L, int NT>
__device__ __forceinline__ void bn_store(BnTensor t, int64_t row, int d, int tid, const float (&v)[8])
{
    if constexpr (L == BN_8) {
        if (tid * 8 < d) {
            if (t.bf16) {
                *reinterpret_cast<u32x4 *>((__bf16 *)t.p + row * d + (uint32_t)(tid * 8)) =
                    u32x4{bn_pack(v[0], v[1]), bn_pack(v[2], v[3]), bn_pack(v[4], v[5]), bn_pack(v[6], v[7])};
            } else {
                float *q = (float *)t.p + row * d + (uint32_t)(tid * 8);
                *reinterpret_cast<float4 *>(q) = make_float4(v[0], v[1], v[2], v[3]);
                *reinterpret_cast<float4 *>(q + 4) = make_float4(v[4], v[5], v[6], v[7]);
            }
        }
    } else if constexpr (L == BN_END) {
        if (tid * 8 < d) {
            const uint32_t c = bn_end(tid, d);
            if (t.bf16) {
                *reinterpret_cast<u32x4_al2 *>((__bf16 *)t.p + row * d + c) =
                    u32x4_al2{bn_pack(v[0], v[1]), bn_pack(v[2], v[3]), bn_pack(v[4], v[5]), bn_pack(v[6], v[7])};
            } else {
                float *q = (float *)t.p + row * d + c;
#pragma unroll
                for (int h = 0; h < 8; h += 4)
                    *reinterpret_cast<u32x4_al4 *>(q + h) = u32x4_al4{__float_as_uint(v[h]), __float_as_uint(v[h + 1]),
                                                                      __float_as_uint(v[h + 2]), __float_as_uint(v[h + 3])};
            }
        }
    } else if constexpr (L == BN_4) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = h * 4 * NT + tid * 4;
            if (c < d) {
                if (t.bf16)
                    *reinterpret_cast<uint2 *>((__bf16 *)t.p + row * d + c) =
                        make_uint2(bn_pack(v[4 * h], v[4 * h + 1]), bn_pack(v[4 * h + 2], v[4 * h + 3]));
                else
                    *reinterpret_cast<float4 *>((float *)t.p + row * d + c) =
                        make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
            }
        }
    } else {
        bn_forget(tid);
        if (t.bf16) {
            __bf16 *q = (__bf16 *)t.p + row * d;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e * NT + tid < d)
                    q[(uint32_t)(e * NT + tid)] = (__bf16)v[e];
        } else {
            float *q = (float *)t.p + row * d;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e * NT + tid < d)
                    q[(uint32_t)(e * NT + tid)] = v[e];
        }
    }
}

// Weights of a row's columns, `none` where the pointer is NULL.  Columns past d
// hold 0 everywhere in a row, weights and biases too, so they add nothing to a sum.
template <BnLay L, int NT>
__device__ __forceinline__ void bn_weights(BnTensor t, int d, int tid, float none, float (&w)[8])
{
    if (t.p) {
        bn_values(bn_load<L, NT>(t, 0, d, tid), t.bf16, w);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            w[e] = none;
    }
}

// Sum over a row's NT < 64 lanes: pairs, quads, halves of 16 and 16 lanes by DPP,
// the two 16s of a row of 32 lanes by a shuffle.  The same bits in every lane.
template <int NT> __device__ __forceinline__ float bn_lanes_sum(float v)
{
    auto dpp = [](float x, auto ctrl) {
        return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), decltype(ctrl)::value, 0xf, 0xf, false));
    };
    v += dpp(v, std::integral_constant<int, 0xB1>{});  // quad_perm 1 0 3 2
    if constexpr (NT >= 4)
        v += dpp(v, std::integral_constant<int, 0x4E>{});  // quad_perm 2 3 0 1
    if constexpr (NT >= 8)
        v += dpp(v, std::integral_constant<int, 0x141>{});  // row_half_mirror
    if constexpr (NT >= 16)
        v += dpp(v, std::integral_constant<int, 0x140>{});  // row_mirror
    if constexpr (NT >= 32)
        v += __shfl_xor(v, 16, 64);
    return v;
}

// Rows that a wave holds side by side, and sums over them, column by column.
template <int NT> constexpr int bn_wave_rows() { return NT < 64 ? 64 / NT : 1; }
template <int NT> __device__ __forceinline__ void bn_rows_sum(float (&v)[8])
{
#pragma unroll
    for (int o = NT; o < 64; o *= 2)
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] += __shfl_xor(v[e], o, 64);
}

// Sums of N values over the NT threads of a row, the same in every thread.
// `slot` alternates between two LDS areas, so one barrier a sum is enough.
template <int NT, int N> __device__ __forceinline__ void row_sums(float (&v)[N], float *red, int &slot)
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = NT < 64 ? bn_lanes_sum<NT < 64 ? NT : 2>(v[i]) : wave_sum(v[i]);
    if constexpr (NT > 64) {
        constexpr int NW = NT / 64;
        float *r = red + slot * (NW * 2);
        slot ^= 1;
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                r[(threadIdx.x >> 6) * N + i] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float s = r[i];
#pragma unroll
            for (int w = 1; w < NW; ++w)
                s += r[w * N + i];
            v[i] = s;
        }
    }
}

// v := vhat; returns rstd.  Columns past d hold 0 on entry and on return.
template <bool LAYER, BnLay L, int NT>
__device__ __forceinline__ float bn_hat(float (&v)[8], int d, int tid, float eps, float *red, int &slot)
{
    const float inv_d = 1.f / (float)d;
    float s[1];
    if constexpr (LAYER) {
        s[0] = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            s[0] += bn_once<L>(v[e], tid, e, d);
        row_sums<NT, 1>(s, red, slot);
        const float mean = s[0] * inv_d;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = bn_in<L, NT>(tid, e, d) ? v[e] - mean : 0.f;
    }
    s[0] = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        s[0] += bn_once<L>(v[e] * v[e], tid, e, d);
    row_sums<NT, 1>(s, red, slot);
    const float rstd = 1.f / sqrtf(s[0] * inv_d + eps);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        v[e] *= rstd;
    return rstd;
}

// g (gradient times weight, 0 past d) := the norm's input gradient.
template <bool LAYER, BnLay L, int NT>
__device__ __forceinline__ void bn_hat_grad(float (&g)[8], const float (&hat)[8], float rstd, int d, int tid,
                                            float *red, int &slot)
{
    float s[LAYER ? 2 : 1];
#pragma unroll
    for (int i = 0; i < (LAYER ? 2 : 1); ++i)
        s[i] = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        s[0] += bn_once<L>(g[e] * hat[e], tid, e, d);
        if constexpr (LAYER)
            s[1] += bn_once<L>(g[e], tid, e, d);
    }
    row_sums<NT>(s, red, slot);
    const float inv_d = 1.f / (float)d, m0 = s[0] * inv_d;
    float m1 = 0.f;
    if constexpr (LAYER)
        m1 = s[1] * inv_d;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        g[e] = (g[e] - m1 - hat[e] * m0) * rstd;
}

// Rows of up to 64 threads share a workgroup of 256 (no LDS), narrow ones a wave
// too; wider rows have a workgroup each.
template <int NT> constexpr int bn_threads() { return NT <= 64 ? 256 : NT; }

template <bool LAYER, BnLay L, int NT>
__global__ __launch_bounds__(bn_threads<NT>()) void block_norm_kernel(BnArgs a)
{
    constexpr int RPW = bn_threads<NT>() / NT;
    __shared__ float red[NT > 64 ? 4 * (NT / 64) : 1];
    int slot = 0;
    const int tid = threadIdx.x % NT;
    const int64_t step = (int64_t)gridDim.x * RPW;
    // (a wave's threads have the same row: known as such, its address is scalar)
    const int first = RPW > 1 ? (int)threadIdx.x / NT : 0;
    int64_t row = (int64_t)blockIdx.x * RPW + (NT == 64 ? __builtin_amdgcn_readfirstlane(first) : first);
    if (row >= a.T)  // whole rows' threads: the sums stay within them
        return;
    const bool block = a.y.p, next = a.n.p;
    Raw8 rr{}, ry{}, rg{};
    auto request = [&](int64_t t) {
        rr = bn_load<L, NT>(a.res, t, a.d, tid);
        if (block)
            ry = bn_load<L, NT>(a.y, t, a.d, tid);
        if (a.gate_span)
            rg = bn_load<L, NT>(a.gate, (int)t / a.gate_span, a.d, tid);
    };
    request(row);
    float wpost[8], bpost[8], wpre[8], bpre[8];
    bn_weights<L, NT>(a.w_post, a.d, tid, 1.f, wpost);
    bn_weights<L, NT>(a.b_post, a.d, tid, 0.f, bpost);
    bn_weights<L, NT>(a.w_pre, a.d, tid, 1.f, wpre);
    bn_weights<L, NT>(a.b_pre, a.d, tid, 0.f, bpre);
    for (; row < a.T; row += step) {
        float r[8], p[8], g[8];
        bn_values(rr, a.res.bf16, r);
        bn_values(ry, a.y.bf16, p);
        bn_values(rg, a.gate.bf16, g);
        if (row + step < a.T)  // on its way while this row's sums are taken
            request(row + step);
        if (block) {
            if (a.post) {
                bn_hat<LAYER, L, NT>(p, a.d, tid, a.eps, red, slot);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    p[e] = p[e] * wpost[e] + bpost[e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
                r[e] += a.alpha * (a.gate_span ? p[e] * g[e] : p[e]);
            if (a.out.p)
                bn_store<L, NT>(a.out, row, a.d, tid, r);
        }
        if (next) {
            bn_hat<LAYER, L, NT>(r, a.d, tid, a.eps, red, slot);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                r[e] = r[e] * wpre[e] + bpre[e];
            bn_store<L, NT>(a.n, row, a.d, tid, r);
        }
    }
}

// Row group b (the NT threads of a row, or a wave of several rows; 4 waves in a
// workgroup when NT <= 64) takes the rows [b rows, (b + 1) rows), a wave of several
// that many at a step.  Its sums over those rows stay in
// registers and leave as one partial row per vector.  A gate row whose rows all
// lie in the group is finished here; one cut at the group's first row leaves in
// slot 4, one cut at its last row only in slot 5.
template <bool LAYER, bool BIAS, BnLay L, int NT>
__global__ __launch_bounds__(bn_threads<NT>()) void block_norm_backward_kernel(BnArgs a)
{
    __shared__ float red[NT > 64 ? 4 * (NT / 64) : 1];
    int slot = 0;
    const int tid = threadIdx.x % NT;
    constexpr int K = bn_wave_rows<NT>();
    const int seg = K > 1 ? (int)(threadIdx.x & 63) / NT : 0;
    const int grp = NT <= 64 ? (int)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / 64) : (int)blockIdx.x;
    if (grp >= a.groups)
        return;
    const int64_t r0 = (int64_t)grp * a.rows;
    const int64_t r1 = r0 + a.rows < a.T ? r0 + a.rows : a.T;
    float wpost[8], bpost[8], wpre[8], acc[4][8], ag[8];
    // 1024 threads have 128 registers each: where the weights do not fit in them they come again for every row (2048
    // x 8192: layer norm with biases 162 -> 127 us, RMS in bf16 93 -> 76; where they do fit, 98 us and 105 so)
    constexpr bool HOLD = NT < 1024 || (L == BN_4 && !LAYER && !BIAS);
    auto weights = [&](BnTensor t, float none, float (&w)[8]) {
        int again = tid;
        if constexpr (!HOLD)
            bn_forget(again);
        bn_weights<L, NT>(t, a.d, again, none, w);
    };
    if constexpr (HOLD) {
        weights(a.w_post, 1.f, wpost);
        weights(a.b_post, 0.f, bpost);
        weights(a.w_pre, 1.f, wpre);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        ag[e] = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            acc[k][e] = 0.f;
    }
    int64_t group = a.gate_span ? (int)r0 / a.gate_span : 0;  // the gate row that ag belongs to
    for (int64_t base = r0; base < r1; base += K) {
        const int64_t row = base + seg;
        float gp[8];  // this row's part of the gate's gradient, of rows side by side
        if constexpr (K > 1) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                gp[e] = 0.f;
        }
        if (row < r1)
            [&] {
                Raw8 ro{}, rd{}, rn{}, ry{}, rg{};
                if (a.dout.p)
                    rd = bn_load<L, NT, true>(a.dout, row, a.d, tid);
                if (a.dn.p) {
                    ro = bn_load<L, NT, true>(a.res, row, a.d, tid);
                    rn = bn_load<L, NT, true>(a.dn, row, a.d, tid);
                }
                if (a.y.p)
                    ry = bn_load<L, NT, true>(a.y, row, a.d, tid);
                if (a.gate_span)
                    rg = bn_load<L, NT>(a.gate, (int)row / a.gate_span, a.d, tid);
                float dr[8];
                bn_values(rd, a.dout.bf16, dr);
                if (a.dn.p) {
                    float hat[8], dn[8];
                    bn_values(ro, a.res.bf16, hat);
                    bn_values(rn, a.dn.bf16, dn);
                    const float rstd = bn_hat<LAYER, L, NT>(hat, a.d, tid, a.eps, red, slot);
                    if constexpr (!HOLD)
                        weights(a.w_pre, 1.f, wpre);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        acc[2][e] += dn[e] * hat[e];
                        if constexpr (BIAS)
                            acc[3][e] += dn[e];
                        dn[e] *= wpre[e];
                    }
                    bn_hat_grad<LAYER, L, NT>(dn, hat, rstd, a.d, tid, red, slot);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        dr[e] += dn[e];
                }
                bn_store<L, NT>(a.dres, row, a.d, tid, dr);
                if (!a.y.p)
                    return;
                float hat[8], rstd = 1.f;
                bn_values(ry, a.y.bf16, hat);
                if (a.post)
                    rstd = bn_hat<LAYER, L, NT>(hat, a.d, tid, a.eps, red, slot);
                if constexpr (!HOLD) {
                    weights(a.w_post, 1.f, wpost);
                    weights(a.b_post, 0.f, bpost);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    dr[e] = bn_in<L, NT>(tid, e, a.d) ? dr[e] * a.alpha : 0.f;
                if (a.gate_span) {
                    float g[8];
                    bn_values(rg, a.gate.bf16, g);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float p = dr[e] * (a.post ? hat[e] * wpost[e] + bpost[e] : hat[e]);
                        if constexpr (K > 1)
                            gp[e] = p;
                        else
                            ag[e] += p;
                        dr[e] *= g[e];
                    }
                }
                if (a.post) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        acc[0][e] += dr[e] * hat[e];
                        if constexpr (BIAS)
                            acc[1][e] += dr[e];
                        dr[e] *= wpost[e];
                    }
                    bn_hat_grad<LAYER, L, NT>(dr, hat, rstd, a.d, tid, red, slot);
                }
                bn_store<L, NT>(a.dy, row, a.d, tid, dr);
            }();
        if (!a.gate_span)
            continue;
        if (K > 1 && a.gate_span == 1) {
            if (row < r1)
                bn_store<L, NT>(a.dgate, row, a.d, tid, gp);
            continue;
        }
        // the gate rows that these rows belong to, each left when its last row in the group has been added
        const int64_t end = base + K < r1 ? base + K : r1;
        const int64_t stop = end < r1 ? (int)end / a.gate_span : (int64_t)(int)(r1 - 1) / a.gate_span + 1;
        const int mine = K > 1 ? (int)row / a.gate_span : 0;
        while (true) {
            if constexpr (K > 1) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    ag[e] += mine == group ? gp[e] : 0.f;
            }
            if (group == stop)
                break;
            bn_rows_sum<NT>(ag);
            const bool head = group * a.gate_span < r0;
            const bool tail = (group + 1) * a.gate_span > r1 && r1 < a.T;
            const BnTensor t = head || tail ? BnTensor{a.part + ((int64_t)(head ? 4 : 5) * a.groups + grp) * bn_pitch(a.d), 0} : a.dgate;
            if (seg == 0)
                bn_store<L, NT>(t, head || tail ? 0 : group, a.d, tid, ag);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                ag[e] = 0.f;
            ++group;
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (a.dw[k]) {
            const BnTensor t{a.part + ((int64_t)k * a.groups + grp) * bn_pitch(a.d), 0};
            bn_rows_sum<NT>(acc[k]);
            if (seg == 0)
                bn_store<L, NT>(t, 0, a.d, tid, acc[k]);
        }
}

// Column sums over the row groups' partial rows in a fixed order: 32 columns a
// workgroup, 32 threads of 4 columns each for them.  blockIdx.y < 4: a weight gradient.  Above: the gate rows that
// are cut between groups, found from the gate rows or from the groups' boundaries,
// whichever are fewer (a.cuts of them, dealt out over the rest of grid y).
__global__ __launch_bounds__(256) void block_norm_reduce_kernel(BnArgs a)
{
    __shared__ __attribute__((aligned(16))) float red[32][32];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), seg = threadIdx.x >> 5;
    auto column = [&](int kind0, int b0, int kind, int b1) {  // partial rows b0 (of kind0), then b0 + 1 .. b1 - 1
        const int n = b1 - b0;
        __syncthreads();
        const int c4 = (threadIdx.x & 7) * 4, s4 = threadIdx.x >> 3;
        float4 p = make_float4(0.f, 0.f, 0.f, 0.f);
        if (blockIdx.x * 32 + c4 < a.d) {
#pragma unroll 8
            for (int i = s4; i < n; i += 32) {
                const float4 v = *reinterpret_cast<const float4 *>(
                    a.part + ((int64_t)(i == 0 ? kind0 : kind) * a.groups + b0 + i) * bn_pitch(a.d) + blockIdx.x * 32 + c4);
                p.x += v.x;
                p.y += v.y;
                p.z += v.z;
                p.w += v.w;
            }
        }
        *reinterpret_cast<float4 *>(&red[s4][c4]) = p;
        __syncthreads();
        float s = 0.f;
        if (seg == 0) {
#pragma unroll
            for (int k = 0; k < 32; ++k)
                s += red[k][threadIdx.x];
        }
        return s;
    };
    if (blockIdx.y < 4) {
        float *dw = a.dw[blockIdx.y];
        if (!dw)
            return;
        const float s = column(blockIdx.y, 0, blockIdx.y, a.groups);
        if (seg == 0 && c < a.d)
            dw[c] = s;
        return;
    }
    for (int k = (int)blockIdx.y - 4; k < a.cuts; k += gridDim.y - 4) {
        int g;
        if (a.gate_span >= a.rows) {
            g = k;
        } else {  // the gate row that boundary k | k + 1 falls into
            g = (k + 1) * a.rows / a.gate_span;
            if (g * a.gate_span == (k + 1) * a.rows)
                continue;
        }
        const int r0 = g * a.gate_span, r1 = a.T - r0 > a.gate_span ? r0 + a.gate_span : a.T;
        const int b0 = r0 / a.rows, b1 = (r1 + a.rows - 1) / a.rows;
        if (b1 - b0 < 2)  // whole inside one group
            continue;
        // begun in group b0 and cut at its end, then at the first row of those that follow; where it begins with a
        // group it is cut at that group's end too
        const float s = column(5, b0, 4, b1);
        if (seg == 0 && c < a.d) {
            if (a.dgate.bf16)
                ((__bf16 *)a.dgate.p)[(int64_t)g * a.d + c] = (__bf16)s;
            else
                ((float *)a.dgate.p)[(int64_t)g * a.d + c] = s;
        }
    }
}

// The threads of a row, and how many rows a wave holds at once.  Narrow rows side
// by side: 65536 rows of 64 take 9 us forward in bf16 (29 us with a wave for each) and
// 36 backward with fp32 streams (95), 262144 rows of 16 take 9 (101) and 36 (302).
static int bn_row_threads(int d)
{
    return d <= 16 ? 2 : d <= 32 ? 4 : d <= 64 ? 8 : d <= 128 ? 16 : d <= 256 ? 32 : d <= 512 ? 64 : d <= 1024 ? 128 : d <= 2048 ? 256 : d <= 4096 ? 512 : 1024;
}
static int bn_rows_at_once(int d) { return bn_row_threads(d) < 64 ? 64 / bn_row_threads(d) : 1; }

// Row groups of the backward pass: about three workgroups of 256 threads per CU,
// as many as its registers allow; each adds up its own rows' weight gradients.
struct BnSteps {
    int steps, most, full;  // a wave's or a workgroup's steps; groups for all registers, and for a workgroup per CU
};
static BnSteps bn_steps(int T, int d)
{
    const int k = bn_rows_at_once(d), threads = bn_row_threads(d) * k;
    return BnSteps{(T + k - 1) / k, BN_BWD_THREADS / threads, 256 * 256 / threads};
}
int block_norm_groups(int T, int d)
{
    const auto [steps, most, full] = bn_steps(T, d);
    int per = (steps + most - 1) / most;
    // few rows: up to 4 steps a group, until there is a workgroup of 256 threads per CU; each group costs a partial
    // row per vector (777 x 1001: 28 us at 195 groups, 24 at 389, 28 at 777)
    const int few = (steps + full - 1) / full < 4 ? (steps + full - 1) / full : 4;
    per = per > few ? per : few;
    return per > 0 ? (steps + per - 1) / per : 0;
}

// One step a group up to `full` groups, then no more until 4 steps each, then 4
// steps a group up to `most`: what the rule above stays below.
int block_norm_most_groups(int T, int d)
{
    const auto [steps, most, full] = bn_steps(T, d);
    if (steps <= 4 * full)
        return steps < full ? steps : full;
    return (steps + 3) / 4 < most ? (steps + 3) / 4 : most;
}

// Whole steps (that a wave holds at once), so that (groups - 1) of them end before row T.
int block_norm_rows(int T, int d)
{
    const int groups = block_norm_groups(T, d), k = bn_rows_at_once(d);
    return groups ? ((T + groups - 1) / groups + k - 1) / k * k : 0;
}

// Workgroups of the forward pass: enough to fill the GPU; rows beyond that come
// one after another with the weights in registers.
constexpr int BN_FWD_THREADS = 256 * 2048;

template <bool LAYER, BnLay L> static hipError_t bn_go(const BnArgs &a, bool backward, hipStream_t s)
{
    auto go = [&](auto nt) {
        constexpr int NT = decltype(nt)::value;
        constexpr int threads = bn_threads<NT>(), per = threads / NT, most = BN_FWD_THREADS / threads;
        if (backward) {
            constexpr int groups = NT <= 64 ? 4 : 1;
            const dim3 grid((a.groups + groups - 1) / groups);
            if (a.dw[1] || a.dw[3])
                block_norm_backward_kernel<LAYER, true, L, NT><<<grid, dim3(threads), 0, s>>>(a);
            else
                block_norm_backward_kernel<LAYER, false, L, NT><<<grid, dim3(threads), 0, s>>>(a);
        } else {
            const int wgs = (int)(((int64_t)a.T + per - 1) / per);
            block_norm_kernel<LAYER, L, NT><<<dim3(wgs < most ? wgs : most), dim3(threads), 0, s>>>(a);
        }
        return hipGetLastError();
    };
    if constexpr (L == BN_ANY)
        return go(std::integral_constant<int, 2>{});
    else
    switch (bn_row_threads(a.d)) {
    case 2:
        return go(std::integral_constant<int, 2>{});
    case 4:
        return go(std::integral_constant<int, 4>{});
    case 8:
        return go(std::integral_constant<int, 8>{});
    case 16:
        return go(std::integral_constant<int, 16>{});
    case 32:
        return go(std::integral_constant<int, 32>{});
    case 64:
        return go(std::integral_constant<int, 64>{});
    case 128:
        return go(std::integral_constant<int, 128>{});
    case 256:
        return go(std::integral_constant<int, 256>{});
    case 512:
        return go(std::integral_constant<int, 512>{});
    default:
        return go(std::integral_constant<int, 1024>{});
    }
}

static hipError_t bn_dispatch(const BnArgs &a, bool layer, bool vec, bool backward, hipStream_t s)
{
    int wide = 0, narrow = 0;  // tensors of rows in fp32 and in bf16
    for (const BnTensor *t : {&a.res, &a.y, &a.out, &a.n, &a.dout, &a.dn, &a.dres, &a.dy})
        if (t->p)
            ++(t->bf16 ? narrow : wide);
    // (narrow rows too: BN_8 would leave half of the threads idle)
    const BnLay lay = !vec ? (a.d < 8 ? BN_ANY : BN_END) : wide > narrow || a.d <= 4 * bn_row_threads(a.d) ? BN_4 : BN_8;
    auto go = [&](auto l) {
        return layer ? bn_go<true, decltype(l)::value>(a, backward, s) : bn_go<false, decltype(l)::value>(a, backward, s);
    };
    switch (lay) {
    case BN_ANY:
        return go(std::integral_constant<BnLay, BN_ANY>{});
    case BN_8:
        return go(std::integral_constant<BnLay, BN_8>{});
    case BN_4:
        return go(std::integral_constant<BnLay, BN_4>{});
    default:
        return go(std::integral_constant<BnLay, BN_END>{});
    }
}

hipError_t launch_block_norm(const BnArgs &a, bool layer, bool vec, hipStream_t s)
{
    return bn_dispatch(a, layer, vec, false, s);
}

hipError_t launch_block_norm_backward(const BnArgs &a, bool layer, bool vec, hipStream_t s)
{
    if (a.T > 0) {
        const hipError_t e = bn_dispatch(a, layer, vec, true, s);
        if (e != hipSuccess)
            return e;
    }
    const bool cut = a.gate_span > 1 && a.groups > 1 && a.rows % a.gate_span != 0;
    BnArgs r = a;
    r.cuts = !cut ? 0 : a.gate_span >= a.rows ? (int)(((int64_t)a.T + a.gate_span - 1) / a.gate_span) : a.groups - 1;
    if (!cut && !a.dw[0] && !a.dw[1] && !a.dw[2] && !a.dw[3])
        return hipSuccess;
    // cut gate rows are dealt out over about 8 workgroups per CU (131072 x 32, 20 rows a gate row: 35 us, over 32
    // of them 75)
    const int cols = (a.d + 31) / 32, most = (2048 + cols - 1) / cols;
    block_norm_reduce_kernel<<<dim3(cols, 4 + (r.cuts < most ? r.cuts : most)), dim3(256), 0, s>>>(r);
    return hipGetLastError();
}

}  // namespace twell
