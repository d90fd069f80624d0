// glu.hip -- the dense gated product h = act(x W_g) * (x W_u) and its backward
// pass (twell_glu_forward, twell_glu_backward).
//
// Forward: one matrix product whose B tile interleaves blocks of W_g and W_u
// rows, so a lane's accumulators hold g and u of the same elements and the
// activation, the product and the optional g and u leave from registers; g and
// u never pass through memory on their way to h.
// Backward, from the stored g and u:
//   dg = dh u act'(g), du = dh act(g)            one pass, [T][dg | du]
//   dx = dg W_g + du W_u                         one product, K = 2 F
//   dW_g = dg^T x, dW_u = du^T x                 one product, M = 2 F, K = T
// dg and du are rounded to the element type, as the matrix units take them.
#include "dense_gemm.h"
#include "glu.h"

namespace twell {

// ------------------------------------------------------------------ activations
// act(g) and act'(g).  FAST (bf16 results): exponentials and reciprocals of the
// hardware's own accuracy (1 ulp and |x| 2^-24), and erf by Abramowitz and
// Stegun's formula 7.1.26 (within 1.5e-7).  A NaN stays one under every act.
template <bool FAST> __device__ __forceinline__ float glu_exp(float x) { return FAST ? __expf(x) : expf(x); }
template <bool FAST> __device__ __forceinline__ float glu_rcp(float x) { return FAST ? __builtin_amdgcn_rcpf(x) : 1.f / x; }

// Half the complementary error function at -g / sqrt 2, and exp(-g^2 / 2).
template <bool FAST> __device__ __forceinline__ float glu_phi(float g, float &e)
{
    e = glu_exp<FAST>(-0.5f * g * g);
    if constexpr (FAST) {
        const float t = __builtin_amdgcn_rcpf(1.f + 0.3275911f * 0.70710678f * fabsf(g));
        const float q = 0.5f * e * t *
                        (0.254829592f + t * (-0.284496736f + t * (1.421413741f + t * (-1.453152027f + t * 1.061405429f))));
        return g < 0.f ? q : 1.f - q;
    } else {
        return 0.5f * erfcf(-0.70710678f * g);
    }
}

constexpr float GLU_T1 = 1.5957691216f, GLU_T3 = 0.044715f;  // gelu_tanh(g) = g sigmoid(T1 (g + T3 g^3))

template <bool FAST> __device__ __forceinline__ float glu_act(float g, int act)
{
    if (act == GLU_RELU)
        return g < 0.f ? 0.f : g;
    if (act == GLU_GELU) {
        float e;
        return g * glu_phi<FAST>(g, e);
    }
    const float z = act == GLU_SILU ? g : GLU_T1 * (g + GLU_T3 * g * g * g);
    return g * glu_rcp<FAST>(1.f + glu_exp<FAST>(-z));
}

template <bool FAST> __device__ __forceinline__ float glu_act_grad(float g, int act, float &a)
{
    if (act == GLU_RELU) {
        a = g < 0.f ? 0.f : g;
        return g > 0.f ? 1.f : g <= 0.f ? 0.f : g;
    }
    if (act == GLU_GELU) {
        float e;
        const float phi = glu_phi<FAST>(g, e);
        a = g * phi;
        return phi + 0.39894228f * g * e;
    }
    const float z = act == GLU_SILU ? g : GLU_T1 * (g + GLU_T3 * g * g * g);
    const float s = glu_rcp<FAST>(1.f + glu_exp<FAST>(-z));
    a = g * s;
    const float dz = act == GLU_SILU ? 1.f : GLU_T1 * (1.f + 3.f * GLU_T3 * g * g);
    const float slope = s * (1.f - s);
    return slope == 0.f ? s : s + g * slope * dz;  // far out, where g or dz may be infinite
}

// ------------------------------------------------------------------ forward
template <int BM, int BN, int WM, int WN>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64) __attribute__((amdgpu_waves_per_eu(2, 2))) void
glu_kernel(GluFwd p)
{
    constexpr int DB = WN / 2, NB = DB / 32;
    using Core = DgCore<BM, BN, WM, WN, true, true, DB>;
    __shared__ __attribute__((aligned(16))) char smem[Core::LDS];
    static_assert(Core::NW * dg_stage_bytes<NB>() <= Core::LDS, "the stores' staging fits");
    int mt, nt, split;
    if (!dg_tile(p.tiles, blockIdx.x, mt, nt, split))
        return;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    Core core;
    const int64_t ld = (int64_t)p.d * 2;
    core.a.setup(p.x, p.x, ld, mt * BM, p.T, p.d, 0, wave, lane);
    core.b.setup(p.wg, p.wu, ld, nt * BN, p.F, p.d, 0, wave, lane);
    f32x16 acc[Core::FM][Core::FN];
    core.run(0, p.d >> 6, smem, tid, acc);
    const int m0 = mt * BM + wave / Core::NWN * WM, n0 = nt * (BN / 2) + wave % Core::NWN * DB;
    char *stage = smem + wave * dg_stage_bytes<NB>();
#pragma unroll
    for (int fm = 0; fm < Core::FM; ++fm) {
        auto g = [&](int fn, int i) { return acc[fm][fn][i]; };
        auto u = [&](int fn, int i) { return acc[fm][fn + NB][i]; };
        if (p.g)
            dg_store_rows<NB>(stage, lane, g, (__bf16 *)p.g, p.F, m0 + fm * 32, n0, p.T, p.F);
        if (p.u)
            dg_store_rows<NB>(stage, lane, u, (__bf16 *)p.u, p.F, m0 + fm * 32, n0, p.T, p.F);
        auto h = [&](int fn, int i) { return glu_act<true>(g(fn, i), p.act) * u(fn, i); };
        dg_store_rows<NB>(stage, lane, h, (__bf16 *)p.h, p.F, m0 + fm * 32, n0, p.T, p.F);
    }
}

// Few rows (T <= 16 MB <= 64): bound by reading the weights once.  A workgroup
// takes 8 neurons, i.e. 8 rows of W_g and 8 of W_u as one 16-row operand, and
// copies up to FEW_KS of their K elements into LDS at a time, all in flight at
// once; two workgroups per CU, so one's copies run beside the other's
// products (v_mfma_f32_16x16x32_bf16).  The waves deal out 64-element K chunks
// and their partial products meet in LDS, added in wave order.
constexpr int FEW_KS = 2048;

typedef float f32x4 __attribute__((ext_vector_type(4)));

template <int MB> __global__ __launch_bounds__(256) void glu_few_kernel(GluFwd p)
{
    constexpr int NW = 4, SB = 16 * FEW_KS * 2;
    __shared__ __attribute__((aligned(16))) char sb[SB];
    static_assert(NW * MB * 4 * 64 * 4 <= SB, "the partial products fit");
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n0 = blockIdx.x * 8, r = lane & 15, q = lane >> 4;
    const int64_t ld = (int64_t)p.d * 2;
    const __amdgpu_buffer_rsrc_t wg = dg_rsrc((const char *)p.wg + n0 * ld), wu = dg_rsrc((const char *)p.wu + n0 * ld);
    f32x4 acc[MB];
    const char *xr[MB];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
        acc[mb] = f32x4{0.f, 0.f, 0.f, 0.f};
        const int m = mb * 16 + r;
        xr[mb] = (const char *)p.x + (int64_t)(m < p.T ? m : p.T - 1) * ld;  // rows past T: their results are dropped
    }
    for (int k0 = 0; k0 < p.d; k0 += FEW_KS) {
        const int ks = p.d - k0 < FEW_KS ? p.d - k0 : FEW_KS;  // a multiple of 64
        const int cpr = ks / 8, spr = (cpr + 15) & ~15;        // 16-byte chunks of a row, and its slots in LDS
        for (int s0 = wave * 64; s0 < 16 * spr; s0 += NW * 64) {
            const int slot = s0 + lane, row = slot / spr, sl = slot - row * spr;
            const int ch = (sl & ~15) | ((sl ^ row) & 15);
            const int voff = (row & 7) * (int)ld + k0 * 2 + (ch < cpr ? ch : 0) * 16;
            if (s0 / spr >= 8)  // 8 rows are whole groups of 64 slots
                dma16(wu, sb + s0 * 16, voff, 0);
            else
                dma16(wg, sb + s0 * 16, voff, 0);
        }
        __builtin_amdgcn_s_waitcnt(0x0070);
        wg_barrier();
        for (int kc = wave; kc < ks / 64; kc += NW) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int ch = kc * 8 + half * 4 + q;
                const u32x4 b = *reinterpret_cast<const u32x4 *>(sb + (r * spr + ((ch & ~15) | ((ch ^ r) & 15))) * 16);
#pragma unroll
                for (int mb = 0; mb < MB; ++mb) {
                    const u32x4 a = ldg16(xr[mb] + (k0 + ch * 8) * 2);
                    acc[mb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                                      __builtin_bit_cast(bf16x8, b), acc[mb], 0, 0, 0);
                }
            }
        }
        __syncthreads();
    }
    float *red = reinterpret_cast<float *>(sb);  // [wave][block][register][lane]
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            red[((wave * MB + mb) * 4 + i) * 64 + lane] = acc[mb][i];
    __syncthreads();
    // row m, column c of a block: register m % 4 of lane 16 (m / 4) + c
    for (int e = tid; e < MB * 128; e += 256) {
        const int mb = e >> 7, m = (e >> 3) & 15, c = e & 7;
        if (mb * 16 + m >= p.T)
            continue;
        const int at = (mb * 4 + (m & 3)) * 64 + (m >> 2) * 16 + c;
        float g = 0.f, u = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            g += red[w * MB * 256 + at];
            u += red[w * MB * 256 + at + 8];
        }
        const int64_t o = (int64_t)(mb * 16 + m) * p.F + n0 + c;
        if (p.g)
            ((__bf16 *)p.g)[o] = (__bf16)g;
        if (p.u)
            ((__bf16 *)p.u)[o] = (__bf16)u;
        ((__bf16 *)p.h)[o] = (__bf16)(glu_act<true>(g, p.act) * u);
    }
}

// ------------------------------------------------------------------ backward
// dg and du from g, u, dh: 10 bytes an element (bf16), bound by memory.  Rows T
// to the next multiple of 64 are zeros: they are the K rows that dW's last
// stage reads past T.
template <typename TI> __global__ __launch_bounds__(256) void glu_dact_kernel(GluBwd p, int rows)
{
    constexpr int E = Elt<TI>::PER_CHUNK;
    const int per_row = p.F / E;
    const int64_t n = (int64_t)rows * per_row;
    for (int64_t c = blockIdx.x * 256LL + threadIdx.x; c < n; c += gridDim.x * 256LL) {
        const int64_t t = c / per_row, j = (c - t * per_row) * E;
        u32x4 og{}, ou{};
        if (t < p.T) {
            const int64_t at = t * p.F + j;
            const u32x4 g = ldg16((const TI *)p.g + at), u = ldg16((const TI *)p.u + at), dh = ldg16((const TI *)p.dh + at);
            TI rg[E], ru[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                float a;
                const float da = glu_act_grad<E == 8>(chunk_elem<TI>(g, e), p.act, a);
                const float d = chunk_elem<TI>(dh, e);
                store_elem(rg + e, d * chunk_elem<TI>(u, e) * da);
                store_elem(ru + e, d * a);
            }
            __builtin_memcpy(&og, rg, 16);
            __builtin_memcpy(&ou, ru, 16);
        }
        TI *o = (TI *)p.dgu + t * glu_pitch(p.F) + j;
        *reinterpret_cast<u32x4 *>(o) = og;
        *reinterpret_cast<u32x4 *>(o + p.F) = ou;
    }
}

// One product of the backward pass.  Rows [0, m_turn) of the result go to out,
// the others to out2; with several splits each writes its fp32 part instead.
struct GluMul {
    int M, N, K;             // K in elements; A has zeros up to a multiple of 64 where it is KS
    const void *a, *b, *b2;  // from K index k_turn on, B's rows come from b2
    int64_t lda, ldb;        // bytes
    int k_turn;
    void *out, *out2;
    int m_turn;
    float *part;
    int splits;
    int MT, NT;     // fp32 tiles
    DgTiles tiles;  // bf16 tiles
};

template <int BM, int BN, int WM, int WN, bool A_KC, bool B_KC>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64) __attribute__((amdgpu_waves_per_eu(2, 2))) void
glu_mul_kernel(GluMul p)
{
    using Core = DgCore<BM, BN, WM, WN, A_KC, B_KC>;
    __shared__ __attribute__((aligned(16))) char smem[Core::LDS];
    static_assert(Core::NW * dg_stage_bytes<Core::FN>() <= Core::LDS, "the stores' staging fits");
    int mt, nt, split;
    if (!dg_tile(p.tiles, blockIdx.x, mt, nt, split))
        return;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    Core core;
    const int nk = (p.K + 63) >> 6, per = (nk + p.splits - 1) / p.splits;
    const int k0 = split * per, k1 = k0 + per < nk ? k0 + per : nk;
    core.a.setup(p.a, p.a, p.lda, mt * BM, p.M, nk * 64, nk, wave, lane);
    core.b.setup(p.b, p.b2, p.ldb, nt * BN, p.N, p.K, p.k_turn >> 6, wave, lane);
    f32x16 acc[Core::FM][Core::FN];
    core.run(k0, k1, smem, tid, acc);
    const int m0 = mt * BM + wave / Core::NWN * WM, n0 = nt * BN + wave % Core::NWN * WN;
    if (p.splits > 1) {
#pragma unroll
        for (int fm = 0; fm < Core::FM; ++fm)
#pragma unroll
            for (int fn = 0; fn < Core::FN; ++fn)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int m = m0 + fm * 32 + acc_row(i, lane), n = n0 + fn * 32 + (lane & 31);
                    if (m < p.M && n < p.N)
                        p.part[((int64_t)split * p.M + m) * p.N + n] = acc[fm][fn][i];
                }
        return;
    }
    char *stage = smem + wave * dg_stage_bytes<Core::FN>();
#pragma unroll
    for (int fm = 0; fm < Core::FM; ++fm) {
        const int m = m0 + fm * 32;  // m_turn is a multiple of 64: a block of 32 rows lies on one side
        const bool second = m >= p.m_turn;
        dg_store_rows<Core::FN>(stage, lane, [&](int fn, int i) { return acc[fm][fn][i]; },
                                (__bf16 *)(second ? p.out2 : p.out), p.N, second ? m - p.m_turn : m, n0,
                                second ? p.M - p.m_turn : p.M < p.m_turn ? p.M : p.m_turn, p.N);
    }
}

// out = sum over the splits of their parts, in order; 4 columns a thread.
template <typename TI> __global__ __launch_bounds__(256) void glu_join_kernel(GluMul p)
{
    const int64_t n4 = (int64_t)p.M * p.N / 4, turn = (int64_t)p.m_turn * p.N;
    for (int64_t c = blockIdx.x * 256LL + threadIdx.x; c < n4; c += gridDim.x * 256LL) {
        float4 s = reinterpret_cast<const float4 *>(p.part)[c];
        for (int k = 1; k < p.splits; ++k) {
            const float4 v = reinterpret_cast<const float4 *>(p.part)[k * n4 + c];
            s.x += v.x;
            s.y += v.y;
            s.z += v.z;
            s.w += v.w;
        }
        const int64_t at = c * 4;
        TI *o = at < turn ? (TI *)p.out + at : (TI *)p.out2 + (at - turn);
        store_elem(o, s.x);
        store_elem(o + 1, s.y);
        store_elem(o + 2, s.z);
        store_elem(o + 3, s.w);
    }
}

// ------------------------------------------------------------------ fp32
// 64 x 128 tiles, 4 waves of 32 x 64, v_mfma_f32_32x32x2f32: a lane supplies one
// element, index l % 32 at K index l / 32, so LDS keeps [K][index] rows for both
// layouts and is read without conflicts.  K in steps of 16, two LDS slots, the
// next step's elements on their way in registers meanwhile.
template <int IDX, bool KC, int DB> struct F32Operand {
    static constexpr int V = IDX / 64;  // float4 a thread
    static constexpr int PITCH = IDX + 4;
    const float *base[V];
    int64_t step;
    int k[V], idx[V];
    const float *second[V];
    int turn, K;

    __device__ __forceinline__ void setup(const void *p, const void *p2, int64_t ld, int idx0, int n, int K_, int turn_,
                                          int tid)
    {
        K = K_;
        turn = turn_;
        step = KC ? 16 : 16 * ld;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int u = v * 256 + tid;
            if constexpr (KC) {
                idx[v] = u >> 2;
                k[v] = (u & 3) * 4;
                constexpr int D = DB > 0 ? DB : 1;
                int q = DB > 0 ? idx0 / 2 + idx[v] / (2 * D) * D + idx[v] % D : idx0 + idx[v];
                q = q < n ? q : n - 1;
                base[v] = (const float *)(DB > 0 && ((idx[v] / D) & 1) ? p2 : p) + q * ld + k[v];
                second[v] = base[v];
            } else {
                k[v] = u / (IDX / 4);
                idx[v] = u % (IDX / 4) * 4;
                const int q = idx0 + idx[v] <= n - 4 ? idx0 + idx[v] : n - 4;
                base[v] = (const float *)p + k[v] * ld + q;
                second[v] = (const float *)p2 + k[v] * ld + q;
            }
        }
    }
    __device__ __forceinline__ void load(int kt, float4 (&r)[V]) const
    {
#pragma unroll
        for (int v = 0; v < V; ++v)
            r[v] = kt * 16 + k[v] >= K ? make_float4(0.f, 0.f, 0.f, 0.f)
                                       : *reinterpret_cast<const float4 *>(kt < turn ? base[v] + kt * step
                                                                                     : second[v] + (kt - turn) * step);
    }
    __device__ __forceinline__ void store(float *lds, const float4 (&r)[V]) const
    {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if constexpr (KC) {
                lds[(k[v] + 0) * PITCH + idx[v]] = r[v].x;
                lds[(k[v] + 1) * PITCH + idx[v]] = r[v].y;
                lds[(k[v] + 2) * PITCH + idx[v]] = r[v].z;
                lds[(k[v] + 3) * PITCH + idx[v]] = r[v].w;
            } else {
                *reinterpret_cast<float4 *>(lds + k[v] * PITCH + idx[v]) = r[v];
            }
        }
    }
};

template <bool A_KC, bool B_KC, int DB> struct F32Core {
    static constexpr int BM = 64, BN = 128, SLOT = 16 * (BM + 4) + 16 * (BN + 4);
    F32Operand<BM, A_KC, 0> a;
    F32Operand<BN, B_KC, DB> b;
    __device__ __forceinline__ void run(int k0, int k1, float *smem, int tid, f32x16 (&acc)[2]) const
    {
        const int lane = tid & 63, wave = tid >> 6, wm = wave >> 1, wn = wave & 1;
#pragma unroll
        for (int fn = 0; fn < 2; ++fn)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                acc[fn][i] = 0.f;
        float4 ra[1], rb[2];
        if (k0 < k1) {
            a.load(k0, ra);
            b.load(k0, rb);
        }
        for (int kt = k0; kt < k1; ++kt) {
            float *sa = smem + ((kt - k0) & 1) * SLOT, *sb = sa + 16 * (BM + 4);
            a.store(sa, ra);
            b.store(sb, rb);
            __syncthreads();
            if (kt + 1 < k1) {
                a.load(kt + 1, ra);
                b.load(kt + 1, rb);
            }
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
                const int kk = k + (lane >> 5), col = lane & 31;
                const float av = sa[kk * (BM + 4) + wm * 32 + col];
#pragma unroll
                for (int fn = 0; fn < 2; ++fn)
                    acc[fn] = __builtin_amdgcn_mfma_f32_32x32x2f32(av, sb[kk * (BN + 4) + wn * 64 + fn * 32 + col],
                                                                   acc[fn], 0, 0, 0);
            }
        }
    }
};

__global__ __launch_bounds__(256) void glu_f32_kernel(GluFwd p)
{
    using Core = F32Core<true, true, 32>;
    __shared__ __attribute__((aligned(16))) float smem[2 * Core::SLOT];
    int mt, nt;
    tile_coords(blockIdx.x, p.MT, p.NT, mt, nt);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    Core core;
    core.a.setup(p.x, p.x, p.d, mt * 64, p.T, p.d, p.d, tid);
    core.b.setup(p.wg, p.wu, p.d, nt * 128, p.F, p.d, p.d, tid);
    f32x16 acc[2];
    core.run(0, p.d / 16, smem, tid, acc);
    const int n = nt * 64 + (wave & 1) * 32 + (lane & 31);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int m = mt * 64 + (wave >> 1) * 32 + acc_row(i, lane);
        if (m < p.T && n < p.F) {
            const int64_t o = (int64_t)m * p.F + n;
            const float g = acc[0][i], u = acc[1][i];
            if (p.g)
                ((float *)p.g)[o] = g;
            if (p.u)
                ((float *)p.u)[o] = u;
            ((float *)p.h)[o] = glu_act<false>(g, p.act) * u;
        }
    }
}

template <bool A_KC, bool B_KC> __global__ __launch_bounds__(256) void glu_mul_f32_kernel(GluMul p)
{
    using Core = F32Core<A_KC, B_KC, 0>;
    __shared__ __attribute__((aligned(16))) float smem[2 * Core::SLOT];
    const int tiles = p.MT * p.NT;
    const int split = blockIdx.x / tiles;
    int mt, nt;
    tile_coords(blockIdx.x - split * tiles, p.MT, p.NT, mt, nt);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int nk = (p.K + 15) >> 4, per = (nk + p.splits - 1) / p.splits;
    const int k0 = split * per, k1 = k0 + per < nk ? k0 + per : nk;
    Core core;
    core.a.setup(p.a, p.a, p.lda / 4, mt * 64, p.M, p.K, nk, tid);
    core.b.setup(p.b, p.b2, p.ldb / 4, nt * 128, p.N, p.K, p.k_turn >> 4, tid);
    f32x16 acc[2];
    core.run(k0, k1, smem, tid, acc);
#pragma unroll
    for (int fn = 0; fn < 2; ++fn)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int m = mt * 64 + (wave >> 1) * 32 + acc_row(i, lane);
            const int n = nt * 128 + (wave & 1) * 64 + fn * 32 + (lane & 31);
            if (m >= p.M || n >= p.N)
                continue;
            if (p.splits > 1)
                p.part[((int64_t)split * p.M + m) * p.N + n] = acc[fn][i];
            else if (m < p.m_turn)
                ((float *)p.out)[(int64_t)m * p.N + n] = acc[fn][i];
            else
                ((float *)p.out2)[(int64_t)(m - p.m_turn) * p.N + n] = acc[fn][i];
        }
}

// ------------------------------------------------------------------ host
static int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

hipError_t launch_glu(int vdtype, const GluFwd &args, hipStream_t s)
{
    GluFwd p = args;
    if (vdtype == 0) {
        p.MT = (int)ceil_div(p.T, 64);
        p.NT = (int)ceil_div(p.F, 64);
        glu_f32_kernel<<<dim3(p.MT * p.NT), dim3(256), 0, s>>>(p);
        return hipGetLastError();
    }
    if (p.T <= GLU_FEW) {
        const dim3 grid(p.F / 8);
        switch ((p.T + 15) / 16) {
        case 1:
            glu_few_kernel<1><<<grid, dim3(256), 0, s>>>(p);
            break;
        case 2:
            glu_few_kernel<2><<<grid, dim3(256), 0, s>>>(p);
            break;
        case 3:
            glu_few_kernel<3><<<grid, dim3(256), 0, s>>>(p);
            break;
        default:
            glu_few_kernel<4><<<grid, dim3(256), 0, s>>>(p);
            break;
        }
        return hipGetLastError();
    }
    if (ceil_div(p.T, 256) * ceil_div(p.F, 128) >= 192) {
        p.tiles = dg_tiles(ceil_div(p.T, 256), ceil_div(p.F, 128));
        glu_kernel<256, 256, 64, 128><<<dim3(8 * p.tiles.rows * p.tiles.cols), dim3(512), 0, s>>>(p);
    } else {
        p.tiles = dg_tiles(ceil_div(p.T, 128), ceil_div(p.F, 64));
        glu_kernel<128, 128, 64, 64><<<dim3(8 * p.tiles.rows * p.tiles.cols), dim3(256), 0, s>>>(p);
    }
    return hipGetLastError();
}

// Tiles and splits of a product of the backward pass.
struct MulPlan {
    bool big;
    int splits;
};

static MulPlan mul_plan(int vdtype, int64_t M, int64_t N, int64_t K)
{
    if (M == 0 || N == 0)
        return {false, 1};
    const int64_t stages = ceil_div(K, 64);
    if (vdtype == 1 && ceil_div(M, 256) * ceil_div(N, 256) >= 192)
        return {true, 1};
    const int64_t tiles = vdtype == 1 ? ceil_div(M, 128) * ceil_div(N, 128) : ceil_div(M, 64) * ceil_div(N, 128);
    int splits = 1;
    while (splits < 16 && tiles * splits * 2 <= 512 && stages / (splits * 2) >= 8)
        splits *= 2;
    return {false, splits};
}

static size_t up256_(size_t b) { return (b + 255) & ~(size_t)255; }

GluWs glu_backward_ws(int T, int d, int F, int vdtype)
{
    GluWs w{};
    const size_t es = vdtype == 1 ? 2 : 4;
    w.part = up256_((size_t)ceil_div(T, 64) * 64 * glu_pitch(F) * es);
    const MulPlan dx = mul_plan(vdtype, T, d, 2 * (int64_t)F), dw = mul_plan(vdtype, 2 * (int64_t)F, d, T);
    const size_t a = dx.splits > 1 ? (size_t)dx.splits * T * d * 4 : 0;
    const size_t b = dw.splits > 1 ? (size_t)dw.splits * 2 * F * d * 4 : 0;
    w.bytes = w.part + (a > b ? a : b);
    return w;
}

template <bool A_KC, bool B_KC> static hipError_t mul_go(int vdtype, GluMul p, hipStream_t s)
{
    const MulPlan plan = mul_plan(vdtype, p.M, p.N, p.K);
    p.splits = plan.splits;
    if (vdtype == 0) {
        p.MT = (int)ceil_div(p.M, 64);
        p.NT = (int)ceil_div(p.N, 128);
        glu_mul_f32_kernel<A_KC, B_KC><<<dim3(p.MT * p.NT * p.splits), dim3(256), 0, s>>>(p);
    } else {
        const int tile = plan.big ? 256 : 128;
        p.tiles = dg_tiles(ceil_div(p.M, tile), ceil_div(p.N, tile));
        const dim3 grid(8 * p.tiles.rows * p.tiles.cols * p.splits);
        if (plan.big)
            glu_mul_kernel<256, 256, 64, 128, A_KC, B_KC><<<grid, dim3(512), 0, s>>>(p);
        else
            glu_mul_kernel<128, 128, 64, 64, A_KC, B_KC><<<grid, dim3(256), 0, s>>>(p);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1)
        return e;
    const int64_t wgs = ceil_div((int64_t)p.M * p.N / 4, 256);
    const dim3 join((unsigned)(wgs < 4096 ? wgs : 4096));
    if (vdtype == 1)
        glu_join_kernel<__bf16><<<join, dim3(256), 0, s>>>(p);
    else
        glu_join_kernel<float><<<join, dim3(256), 0, s>>>(p);
    return hipGetLastError();
}

hipError_t launch_glu_backward(int vdtype, const GluBwd &p, hipStream_t s)
{
    const int es = vdtype == 1 ? 2 : 4;
    const int rows = (int)ceil_div(p.T, 64) * 64;
    hipError_t e;
    if (rows > 0) {
        const int64_t wgs = ceil_div((int64_t)rows * p.F * es / 16, 256);
        const dim3 grid((unsigned)(wgs < 8192 ? wgs : 8192));
        if (vdtype == 1)
            glu_dact_kernel<__bf16><<<grid, dim3(256), 0, s>>>(p, rows);
        else
            glu_dact_kernel<float><<<grid, dim3(256), 0, s>>>(p, rows);
        if ((e = hipGetLastError()) != hipSuccess)
            return e;
    }
    GluMul m{};
    m.a = p.dgu;
    m.lda = glu_pitch(p.F) * es;
    m.ldb = (int64_t)p.d * es;
    m.N = p.d;
    m.part = p.part;
    if (p.dx && p.T > 0) {
        m.M = p.T;
        m.K = 2 * p.F;
        m.b = p.wg;
        m.b2 = p.wu;
        m.k_turn = p.F;
        m.out = m.out2 = p.dx;
        m.m_turn = (int)ceil_div(p.T, 64) * 64;
        if ((e = mul_go<true, false>(vdtype, m, s)) != hipSuccess)
            return e;
    }
    if (p.dwg) {
        m.M = 2 * p.F;
        m.K = p.T;
        m.b = m.b2 = p.x;
        m.k_turn = 1 << 30;
        m.out = p.dwg;
        m.out2 = p.dwu;
        m.m_turn = p.F;
        return mul_go<false, false>(vdtype, m, s);
    }
    return hipSuccess;
}

}  // namespace twell
