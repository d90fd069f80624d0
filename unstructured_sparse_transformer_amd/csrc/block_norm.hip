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
// registers by NT threads of 8 elements (NT = 64 to 1024 by the width), so a
// mean and a variance are two passes over registers, not over memory.  All
// sums are fp32: per thread, then over the wave by DPP, then over the waves
// through LDS.
#include "block_norm.h"
#include "twell_device.h"
#include "wave_ops.h"

#include <type_traits>

namespace twell {

// 8 elements of a row as they lie in memory, requested now and used later.
struct Raw8 {
    u32x4 a, b;
};

// Element e of thread `tid` is column tid * 8 + e (VEC) or e * NT + tid.
template <bool VEC, int NT> __device__ __forceinline__ int bn_col(int tid, int e) { return VEC ? tid * 8 + e : e * NT + tid; }

template <bool VEC, int NT> __device__ __forceinline__ Raw8 bn_load(BnTensor t, int64_t row, int d, int tid)
{
    Raw8 r{};
    if constexpr (VEC) {
        if (tid * 8 < d) {
            if (t.bf16) {
                r.a = ldg16((const __bf16 *)t.p + row * d + tid * 8);
            } else {
                const float *q = (const float *)t.p + row * d + tid * 8;
                r.a = ldg16(q);
                r.b = ldg16(q + 4);
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = e * NT + tid;
            uint32_t w = 0;
            if (c < d)
                w = t.bf16 ? (uint32_t)((const uint16_t *)t.p)[row * d + c] : ((const uint32_t *)t.p)[row * d + c];
            if (t.bf16) {
                r.a[e >> 1] |= w << (16 * (e & 1));
            } else if (e < 4) {
                r.a[e] = w;
            } else {
                r.b[e - 4] = w;
            }
        }
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

template <bool VEC, int NT>
__device__ __forceinline__ void bn_store(BnTensor t, int64_t row, int d, int tid, const float (&v)[8])
{
    if constexpr (VEC) {
        if (tid * 8 < d) {
            if (t.bf16) {
                *reinterpret_cast<u32x4 *>((__bf16 *)t.p + row * d + tid * 8) =
                    u32x4{bn_pack(v[0], v[1]), bn_pack(v[2], v[3]), bn_pack(v[4], v[5]), bn_pack(v[6], v[7])};
            } else {
                float *q = (float *)t.p + row * d + tid * 8;
                *reinterpret_cast<float4 *>(q) = make_float4(v[0], v[1], v[2], v[3]);
                *reinterpret_cast<float4 *>(q + 4) = make_float4(v[4], v[5], v[6], v[7]);
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = e * NT + tid;
            if (c < d) {
                if (t.bf16)
                    ((__bf16 *)t.p)[row * d + c] = (__bf16)v[e];
                else
                    ((float *)t.p)[row * d + c] = v[e];
            }
        }
    }
}

// Weights of a row's columns, `none` where the pointer is NULL.  Columns past d
// hold 0 everywhere in a row, weights and biases too, so they add nothing to a sum.
template <bool VEC, int NT>
__device__ __forceinline__ void bn_weights(BnTensor t, int d, int tid, float none, float (&w)[8])
{
    if (t.p) {
        bn_values(bn_load<VEC, NT>(t, 0, d, tid), t.bf16, w);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            w[e] = none;
    }
}

// Sums of N values over the NT threads of a row, the same in every thread.
// `slot` alternates between two LDS areas, so one barrier a sum is enough.
template <int NT, int N> __device__ __forceinline__ void row_sums(float (&v)[N], float *red, int &slot)
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = wave_sum(v[i]);
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
template <bool LAYER, bool VEC, int NT>
__device__ __forceinline__ float bn_hat(float (&v)[8], int d, int tid, float eps, float *red, int &slot)
{
    const float inv_d = 1.f / (float)d;
    float s[1];
    if constexpr (LAYER) {
        s[0] = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            s[0] += v[e];
        row_sums<NT, 1>(s, red, slot);
        const float mean = s[0] * inv_d;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = bn_col<VEC, NT>(tid, e) < d ? v[e] - mean : 0.f;
    }
    s[0] = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        s[0] += v[e] * v[e];
    row_sums<NT, 1>(s, red, slot);
    const float rstd = 1.f / sqrtf(s[0] * inv_d + eps);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        v[e] *= rstd;
    return rstd;
}

// g (gradient times weight, 0 past d) := the norm's input gradient.
template <bool LAYER, bool VEC, int NT>
__device__ __forceinline__ void bn_hat_grad(float (&g)[8], const float (&hat)[8], float rstd, int d, int tid,
                                            float *red, int &slot)
{
    float s[LAYER ? 2 : 1];
#pragma unroll
    for (int i = 0; i < (LAYER ? 2 : 1); ++i)
        s[i] = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        s[0] += g[e] * hat[e];
        if constexpr (LAYER)
            s[1] += g[e];
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

// Rows of NT = 64 threads share a workgroup of 4 (no LDS); wider rows have a
// workgroup each.
template <int NT> constexpr int bn_threads() { return NT == 64 ? 256 : NT; }

template <bool LAYER, bool VEC, int NT>
__global__ __launch_bounds__(bn_threads<NT>()) void block_norm_kernel(BnArgs a)
{
    constexpr int RPW = bn_threads<NT>() / NT;
    __shared__ float red[NT > 64 ? 4 * (NT / 64) : 1];
    int slot = 0;
    const int tid = threadIdx.x % NT;
    const int64_t row = (int64_t)blockIdx.x * RPW + threadIdx.x / NT;
    if (row >= a.T)  // whole waves: a row is a multiple of 64 threads
        return;
    const Raw8 rr = bn_load<VEC, NT>(a.res, row, a.d, tid);
    float r[8];
    if (a.y.p) {
        const Raw8 ry = bn_load<VEC, NT>(a.y, row, a.d, tid);
        Raw8 rg{};
        if (a.gate_span)
            rg = bn_load<VEC, NT>(a.gate, (int)row / a.gate_span, a.d, tid);
        float p[8];
        bn_values(ry, a.y.bf16, p);
        if (a.post) {
            float w[8], b[8];
            bn_weights<VEC, NT>(a.w_post, a.d, tid, 1.f, w);
            bn_weights<VEC, NT>(a.b_post, a.d, tid, 0.f, b);
            bn_hat<LAYER, VEC, NT>(p, a.d, tid, a.eps, red, slot);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                p[e] = p[e] * w[e] + b[e];
        }
        if (a.gate_span) {
            float g[8];
            bn_values(rg, a.gate.bf16, g);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                p[e] *= g[e];
        }
        bn_values(rr, a.res.bf16, r);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            r[e] += a.alpha * p[e];
        if (a.out.p)
            bn_store<VEC, NT>(a.out, row, a.d, tid, r);
    } else {
        bn_values(rr, a.res.bf16, r);
    }
    if (a.n.p) {
        float w[8], b[8];
        bn_weights<VEC, NT>(a.w_pre, a.d, tid, 1.f, w);
        bn_weights<VEC, NT>(a.b_pre, a.d, tid, 0.f, b);
        bn_hat<LAYER, VEC, NT>(r, a.d, tid, a.eps, red, slot);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            r[e] = r[e] * w[e] + b[e];
        bn_store<VEC, NT>(a.n, row, a.d, tid, r);
    }
}

// Workgroup b takes the rows [b rows, (b + 1) rows).  Its sums over those rows
// stay in registers and leave as one partial row per vector.  A gate row whose
// rows all lie in the workgroup is finished here; one cut at the workgroup's
// first row leaves in slot 4, one cut at its last row only in slot 5.
template <bool LAYER, bool VEC, int NT>
__global__ __launch_bounds__(NT) void block_norm_backward_kernel(BnArgs a)
{
    __shared__ float red[NT > 64 ? 4 * (NT / 64) : 1];
    int slot = 0;
    const int tid = threadIdx.x;
    const int64_t r0 = (int64_t)blockIdx.x * a.rows;
    const int64_t r1 = r0 + a.rows < a.T ? r0 + a.rows : a.T;
    float wpost[8], bpost[8], wpre[8], acc[4][8], ag[8];
    bn_weights<VEC, NT>(a.w_post, a.d, tid, 1.f, wpost);
    bn_weights<VEC, NT>(a.b_post, a.d, tid, 0.f, bpost);
    bn_weights<VEC, NT>(a.w_pre, a.d, tid, 1.f, wpre);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        ag[e] = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            acc[k][e] = 0.f;
    }
    int64_t group = a.gate_span ? (int)r0 / a.gate_span : 0;
    for (int64_t row = r0; row < r1; ++row) {
        Raw8 ro{}, rd{}, rn{}, ry{}, rg{};
        if (a.dout.p)
            rd = bn_load<VEC, NT>(a.dout, row, a.d, tid);
        if (a.dn.p) {
            ro = bn_load<VEC, NT>(a.res, row, a.d, tid);
            rn = bn_load<VEC, NT>(a.dn, row, a.d, tid);
        }
        if (a.y.p)
            ry = bn_load<VEC, NT>(a.y, row, a.d, tid);
        if (a.gate_span)
            rg = bn_load<VEC, NT>(a.gate, (int)row / a.gate_span, a.d, tid);
        float dr[8];
        bn_values(rd, a.dout.bf16, dr);
        if (a.dn.p) {
            float hat[8], dn[8];
            bn_values(ro, a.res.bf16, hat);
            bn_values(rn, a.dn.bf16, dn);
            const float rstd = bn_hat<LAYER, VEC, NT>(hat, a.d, tid, a.eps, red, slot);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                acc[2][e] += dn[e] * hat[e];
                acc[3][e] += dn[e];
                dn[e] *= wpre[e];
            }
            bn_hat_grad<LAYER, VEC, NT>(dn, hat, rstd, a.d, tid, red, slot);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                dr[e] += dn[e];
        }
        bn_store<VEC, NT>(a.dres, row, a.d, tid, dr);
        if (!a.y.p)
            continue;
        float hat[8], rstd = 1.f;
        bn_values(ry, a.y.bf16, hat);
        if (a.post)
            rstd = bn_hat<LAYER, VEC, NT>(hat, a.d, tid, a.eps, red, slot);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            dr[e] = bn_col<VEC, NT>(tid, e) < a.d ? dr[e] * a.alpha : 0.f;
        if (a.gate_span) {
            float g[8];
            bn_values(rg, a.gate.bf16, g);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                ag[e] += dr[e] * (a.post ? hat[e] * wpost[e] + bpost[e] : hat[e]);
                dr[e] *= g[e];
            }
            const int64_t next = (int)(row + 1) / a.gate_span;
            if (next != group || row + 1 == r1) {
                const bool head = group * a.gate_span < r0;
                const bool tail = (group + 1) * a.gate_span > r1 && r1 < a.T;
                if (!head && !tail) {
                    bn_store<VEC, NT>(a.dgate, group, a.d, tid, ag);
                } else {
                    const BnTensor t{a.part + ((int64_t)(head ? 4 : 5) * a.wgs + blockIdx.x) * a.d, 0};
                    bn_store<VEC, NT>(t, 0, a.d, tid, ag);
                }
                group = next;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    ag[e] = 0.f;
            }
        }
        if (a.post) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                acc[0][e] += dr[e] * hat[e];
                acc[1][e] += dr[e];
                dr[e] *= wpost[e];
            }
            bn_hat_grad<LAYER, VEC, NT>(dr, hat, rstd, a.d, tid, red, slot);
        }
        bn_store<VEC, NT>(a.dy, row, a.d, tid, dr);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (a.dw[k]) {
            const BnTensor t{a.part + ((int64_t)k * a.wgs + blockIdx.x) * a.d, 0};
            bn_store<VEC, NT>(t, 0, a.d, tid, acc[k]);
        }
}

// Column sums over the workgroups' partial rows in a fixed order: 32 columns a
// workgroup, 8 threads a column.  blockIdx.y < 4: a weight gradient.  Above:
// the gate rows that are cut between workgroups; the boundaries b - 1 | b are
// dealt out over the rest of grid y, and the first boundary inside a gate row
// owns it.
__global__ __launch_bounds__(256) void block_norm_reduce_kernel(BnArgs a)
{
    __shared__ float red[8][33];
    const int cl = threadIdx.x & 31, seg = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + cl;
    auto column = [&](int kind0, int b0, int kind, int b1) {  // partial rows b0 (of kind0), then b0 + 1 .. b1 - 1
        const int n = b1 - b0;
        float s = 0.f;
        if (c < a.d) {
#pragma unroll 4
            for (int i = seg; i < n; i += 8)
                s += a.part[((int64_t)(i == 0 ? kind0 : kind) * a.wgs + b0 + i) * a.d + c];
        }
        __syncthreads();
        red[seg][cl] = s;
        __syncthreads();
        s = red[0][cl];
#pragma unroll
        for (int k = 1; k < 8; ++k)
            s += red[k][cl];
        return s;
    };
    if (blockIdx.y < 4) {
        float *dw = a.dw[blockIdx.y];
        if (!dw)
            return;
        const float s = column(blockIdx.y, 0, blockIdx.y, a.wgs);
        if (seg == 0 && c < a.d)
            dw[c] = s;
        return;
    }
    for (int b = 1 + (int)blockIdx.y - 4; b < a.wgs; b += gridDim.y - 4) {
        const int64_t first = (int64_t)b * a.rows;  // the first row past the boundary
        const int64_t g = first / a.gate_span, g0 = g * a.gate_span;
        if (g0 >= first || g0 < first - a.rows)  // not cut here, or owned by an earlier boundary
            continue;
        const int64_t g1 = g0 + a.gate_span < a.T ? g0 + a.gate_span : a.T;
        const int b1 = (int)((g1 + a.rows - 1) / a.rows);
        // the row begins inside workgroup b - 1: at its first row it is whole there and cut only at the end
        const float s = column(5, b - 1, 4, b1);
        if (seg == 0 && c < a.d) {
            if (a.dgate.bf16)
                ((__bf16 *)a.dgate.p)[g * a.d + c] = (__bf16)s;
            else
                ((float *)a.dgate.p)[g * a.d + c] = s;
        }
    }
}

int block_norm_wgs(int T)
{
    const int rows = (T + BN_BWD_WGS - 1) / BN_BWD_WGS;
    return rows > 0 ? (T + rows - 1) / rows : 0;
}

template <bool LAYER, bool VEC> static hipError_t bn_go(const BnArgs &a, bool backward, hipStream_t s)
{
    auto go = [&](auto nt) {
        constexpr int NT = decltype(nt)::value;
        if (backward) {
            block_norm_backward_kernel<LAYER, VEC, NT><<<dim3(a.wgs), dim3(NT), 0, s>>>(a);
        } else {
            constexpr int RPW = bn_threads<NT>() / NT;
            block_norm_kernel<LAYER, VEC, NT><<<dim3((a.T + RPW - 1) / RPW), dim3(bn_threads<NT>()), 0, s>>>(a);
        }
        return hipGetLastError();
    };
    if (a.d <= 512)
        return go(std::integral_constant<int, 64>{});
    if (a.d <= 1024)
        return go(std::integral_constant<int, 128>{});
    if (a.d <= 2048)
        return go(std::integral_constant<int, 256>{});
    if (a.d <= 4096)
        return go(std::integral_constant<int, 512>{});
    return go(std::integral_constant<int, 1024>{});
}

static hipError_t bn_dispatch(const BnArgs &a, bool layer, bool vec, bool backward, hipStream_t s)
{
    if (layer)
        return vec ? bn_go<true, true>(a, backward, s) : bn_go<true, false>(a, backward, s);
    return vec ? bn_go<false, true>(a, backward, s) : bn_go<false, false>(a, backward, s);
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
    const bool cut = a.gate_span > 1 && a.wgs > 1 && a.rows % a.gate_span != 0;
    const bool vectors = a.dw[0] || a.dw[1] || a.dw[2] || a.dw[3];
    if (!cut && !vectors)
        return hipSuccess;
    const int bounds = cut ? (a.wgs - 1 < 16 ? a.wgs - 1 : 16) : 0;
    block_norm_reduce_kernel<<<dim3((a.d + 31) / 32, 4 + bounds), dim3(256), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace twell
