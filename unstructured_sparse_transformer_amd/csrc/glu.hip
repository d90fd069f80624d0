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
template <int BM, int BN, int WM, int WN, int S>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64) __attribute__((amdgpu_waves_per_eu(2, 2))) void
glu_kernel(GluFwd p)
{
    constexpr int DB = WN / 2, NB = DB / 32;
    using Core = DgCore<BM, BN, WM, WN, true, true, DB, S>;
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
    const int nk = p.d >> 6, per = (nk + p.splits - 1) / p.splits, k0 = split * per;
    core.run(k0, k0 + per < nk ? k0 + per : nk, smem, tid, acc);
    const int m0 = mt * BM + wave / Core::NWN * WM, n0 = nt * (BN / 2) + wave % Core::NWN * DB;
    if (p.splits > 1) {
#pragma unroll
        for (int fm = 0; fm < Core::FM; ++fm)
#pragma unroll
            for (int fn = 0; fn < Core::FN; ++fn)
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const int m = m0 + fm * 32 + (lane & 31), n = n0 + fn % NB * 32 + acc_row(i, lane);
                    const f32x16 &v = acc[fm][fn];
                    if (m < p.T && n < p.F)
                        *reinterpret_cast<float4 *>(p.part + ((int64_t)(split * 2 + fn / NB) * p.T + m) * p.F + n) =
                            make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                }
        return;
    }
    char *stage = smem + wave * dg_stage_bytes<NB>();
#pragma unroll
    for (int fm = 0; fm < Core::FM; ++fm) {
        auto g = [&](int fn, int i) { return acc[fm][fn][i]; };
        auto u = [&](int fn, int i) { return acc[fm][fn + NB][i]; };
        // g and u wait for the backward pass: past the caches (1-3% of the call)
        if (p.g)
            dg_store_rows<NB, true>(stage, lane, g, (__bf16 *)p.g, p.F, m0 + fm * 32, n0, p.T, p.F);
        if (p.u)
            dg_store_rows<NB, true>(stage, lane, u, (__bf16 *)p.u, p.F, m0 + fm * 32, n0, p.T, p.F);
        auto h = [&](int fn, int i) { return glu_act<true>(g(fn, i), p.act) * u(fn, i); };
        dg_store_rows<NB>(stage, lane, h, (__bf16 *)p.h, p.F, m0 + fm * 32, n0, p.T, p.F);
    }
}

// Few rows: the weights stream through a ring of S LDS slots, one stage (128
// bytes, 64 bf16 or 32 fp32 K elements, of the workgroup's NB rows of W_g, its NB of W_u, and of x) a slot,
// with the copies of S - 1 stages in flight, two workgroups per CU.  Bound by
// reading the weights once: 67 MB of the 2B-like layer in 12.9 us at T = 1
// (5.2 TB/s) and 13.5 us at T = 64.  Workgroups start at different stages:
// W's rows are a power of two apart, and all of them at the same columns meet
// few of the memory channels (17.6 us).  The 4 waves share a stage by K,
// 16 elements each, and their partial products meet in LDS at the end, added in
// wave order.
template <typename TI, int BM, int NB, int S> __global__ __launch_bounds__(256) void glu_stream_kernel(GluFwd p)
{
    constexpr int R = 2 * NB, FM = BM / 32, FN = R / 32;
    constexpr int A_BYTES = BM * 128, SLOT = A_BYTES + R * 128, A_LD = BM / 32, B_LD = R / 32;
    constexpr int RED = 4 * FM * FN * 16 * 64 * 4;
    __shared__ __attribute__((aligned(16))) char smem[S * SLOT > RED ? S * SLOT : RED];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n0 = blockIdx.x * NB;
    const int64_t ld = (int64_t)p.d * sizeof(TI);
    const __amdgpu_buffer_rsrc_t rx = dg_rsrc(p.x), rg = dg_rsrc((const char *)p.wg + n0 * ld),
                                 ru = dg_rsrc((const char *)p.wu + n0 * ld);
    // copy j of a wave fills rows (j 4 + wave) 8 .. + 7; x's rows past T stay as they are (their results are dropped)
    int voff[A_LD + B_LD], na = 0;
#pragma unroll
    for (int j = 0; j < A_LD + B_LD; ++j) {
        const bool x = j < A_LD;
        const int r = ((x ? j : j - A_LD) * 4 + wave) * 8 + (lane >> 3);
        const int c = (lane & 7) ^ ((r >> 1) & 7);
        const int row = x ? (r < p.T ? r : p.T - 1) : r % NB;
        voff[j] = row * (int)ld + c * 16;
        na += x && (j * 4 + wave) * 8 < p.T;
    }
    const int nk = (int)(ld >> 7);
    const int rot = (int)(blockIdx.x % (unsigned)nk);
    auto load = [&](int k, char *slot) {
        const int kt = k + rot < nk ? k + rot : k + rot - nk;
#pragma unroll
        for (int j = 0; j < A_LD; ++j)
            if (j < na)
                dma16(rx, slot + (j * 4 + wave) * 1024, voff[j], kt * 128);
#pragma unroll
        for (int j = 0; j < B_LD; ++j) {
            const int r = (j * 4 + wave) * 8;
            dma16(r < NB ? rg : ru, slot + A_BYTES + r * 128, voff[A_LD + j], kt * 128);
        }
    };
    f32x16 acc[FM][FN];
#pragma unroll
    for (int fm = 0; fm < FM; ++fm)
#pragma unroll
        for (int fn = 0; fn < FN; ++fn)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                acc[fm][fn][i] = 0.f;
#pragma unroll
    for (int k = 0; k < S - 1; ++k)
        if (k < nk)
            load(k, smem + k * SLOT);
    int slot = 0;
    for (int kt = 0; kt < nk; ++kt) {
        // stage kt has arrived: the S - 2 stages after it may be on their way (fewer at the end: then all are waited for)
        if (kt + S - 1 > nk)
            __builtin_amdgcn_s_waitcnt(0x0070);
        else if (na == 0)
            dg_wait<(S - 2) * B_LD>();
        else if (na == 1)
            dg_wait<(S - 2) * (B_LD + 1)>();
        else
            dg_wait<(S - 2) * (B_LD + 2)>();
        wg_barrier();  // and every wave has read stage kt - 1, whose slot is filled again
        if (kt + S - 1 < nk)
            load(kt + S - 1, smem + (slot == 0 ? S - 1 : slot - 1) * SLOT);
        const char *cur = smem + slot * SLOT;
        u32x4 a[FM], b[FN];
#pragma unroll
        for (int f = 0; f < FM; ++f)
            a[f] = DgOperand<32, true, 1>::fragment(cur, f * 32, wave, lane);
#pragma unroll
        for (int f = 0; f < FN; ++f)
            b[f] = DgOperand<32, true, 1>::fragment(cur + A_BYTES, f * 32, wave, lane);
#pragma unroll
        for (int fm = 0; fm < FM; ++fm)
#pragma unroll
            for (int fn = 0; fn < FN; ++fn)
                mfma_chunk(TI{}, a[fm], b[fn], acc[fm][fn]);
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the slot has been read
        slot = slot + 1 == S ? 0 : slot + 1;
    }
    __syncthreads();
    float *red = reinterpret_cast<float *>(smem);  // [wave][block][register][lane]
#pragma unroll
    for (int fm = 0; fm < FM; ++fm)
#pragma unroll
        for (int fn = 0; fn < FN; ++fn)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                red[((wave * FM * FN + fm * FN + fn) * 16 + i) * 64 + lane] = acc[fm][fn][i];
    __syncthreads();
    for (int e = tid; e < BM * NB; e += 256) {
        const int m = e / NB, c = e % NB, r = m & 31;
        if (m >= p.T)
            break;
        // row r of a block: register (r / 8) 4 + r % 4 of the lanes of its half; u's columns follow g's NB
        const int at = ((r >> 3) * 4 + (r & 3)) * 64 + ((r >> 2) & 1) * 32;
        const int bg = (m >> 5) * FN, bu = bg + (NB >> 5);
        float g = 0.f, u = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            g += red[(w * FM * FN + bg) * 1024 + at + c];
            u += red[(w * FM * FN + bu) * 1024 + at + (c + NB) % 32];
        }
        const int64_t o = (int64_t)m * p.F + n0 + c;
        if (p.g)
            store_elem((TI *)p.g + o, g);
        if (p.u)
            store_elem((TI *)p.u + o, u);
        store_elem((TI *)p.h + o, glu_act<sizeof(TI) == 2>(g, p.act) * u);
    }
}

// h (and g, u) from the splits' parts, added in order; 4 columns a thread.
template <typename TI> __global__ __launch_bounds__(256) void glu_join_act_kernel(GluFwd p)
{
    const int64_t n4 = (int64_t)p.T * p.F / 4;
    for (int64_t c = blockIdx.x * 256LL + threadIdx.x; c < n4; c += gridDim.x * 256LL) {
        float v[2][4];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            float4 s = reinterpret_cast<const float4 *>(p.part)[w * n4 + c];
            for (int k = 1; k < p.splits; ++k) {
                const float4 t = reinterpret_cast<const float4 *>(p.part)[(2 * k + w) * n4 + c];
                s.x += t.x;
                s.y += t.y;
                s.z += t.z;
                s.w += t.w;
            }
            v[w][0] = s.x;
            v[w][1] = s.y;
            v[w][2] = s.z;
            v[w][3] = s.w;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (p.g)
                store_elem((TI *)p.g + c * 4 + e, v[0][e]);
            if (p.u)
                store_elem((TI *)p.u + c * 4 + e, v[1][e]);
            store_elem((TI *)p.h + c * 4 + e, glu_act<sizeof(TI) == 2>(v[0][e], p.act) * v[1][e]);
        }
    }
}

// ------------------------------------------------------------------ backward
// dg and du from g, u, dh: 10 bytes an element (bf16), bound by memory (115 us,
// 5.8 TB/s, at 8192 x 8192).  ONCE: the inputs are more than the 256 MB behind the
// L2s keep until here, and are read past the caches (122 us through them; where
// they do fit it is the other way round, 9.3 against 10.0 us at 1003 x 4096).
// Rows T to the next multiple of 64 are zeros: they are the K rows that dW's
// last stage reads past T.
template <bool ONCE> __device__ __forceinline__ u32x4 glu_load(const void *p)
{
    const u32x4 *q = reinterpret_cast<const u32x4 *>(p);
    if constexpr (ONCE)
        return __builtin_nontemporal_load(q);
    return *q;
}

template <typename TI, bool ONCE> __global__ __launch_bounds__(256) void glu_dact_kernel(GluBwd p, int rows)
{
    constexpr int E = Elt<TI>::PER_CHUNK;
    const int per_row = p.F / E;
    const int64_t n = (int64_t)rows * per_row;
    for (int64_t c = blockIdx.x * 256LL + threadIdx.x; c < n; c += gridDim.x * 256LL) {
        const int64_t t = c / per_row, j = (c - t * per_row) * E;
        u32x4 og{}, ou{};
        if (t < p.T) {
            const int64_t at = t * p.F + j;
            const u32x4 g = glu_load<ONCE>((const TI *)p.g + at), u = glu_load<ONCE>((const TI *)p.u + at),
                        dh = glu_load<ONCE>((const TI *)p.dh + at);
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

template <int BM, int BN, int WM, int WN, int S, bool A_KC, bool B_KC>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64) __attribute__((amdgpu_waves_per_eu(2, 2))) void
glu_mul_kernel(GluMul p)
{
    using Core = DgCore<BM, BN, WM, WN, A_KC, B_KC, 0, S>;
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
                for (int i = 0; i < 16; i += 4) {
                    const int m = m0 + fm * 32 + (lane & 31), n = n0 + fn * 32 + acc_row(i, lane);
                    const f32x16 &v = acc[fm][fn];
                    if (m < p.M && n < p.N)
                        *reinterpret_cast<float4 *>(p.part + ((int64_t)split * p.M + m) * p.N + n) =
                            make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
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
// next F32_AHEAD steps' elements on their way in registers meanwhile (one step
// ahead left a load's whole latency to wait for: 59 us at 300 x 1024 x 1024).
constexpr int F32_AHEAD = 4;
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
        float4 ra[F32_AHEAD][1], rb[F32_AHEAD][2];
#pragma unroll
        for (int j = 0; j < F32_AHEAD; ++j)
            if (k0 + j < k1) {
                a.load(k0 + j, ra[j]);
                b.load(k0 + j, rb[j]);
            }
        for (int kt = k0; kt < k1; kt += F32_AHEAD) {
#pragma unroll
            for (int j = 0; j < F32_AHEAD; ++j) {
                if (kt + j >= k1)
                    break;
                float *sa = smem + (j & 1) * SLOT, *sb = sa + 16 * (BM + 4);
                a.store(sa, ra[j]);
                b.store(sb, rb[j]);
                __syncthreads();  // the other slot's readers have passed the barrier before
                if (kt + j + F32_AHEAD < k1) {
                    a.load(kt + j + F32_AHEAD, ra[j]);
                    b.load(kt + j + F32_AHEAD, rb[j]);
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
    }
};

__global__ __launch_bounds__(256) void glu_f32_kernel(GluFwd p)
{
    using Core = F32Core<true, true, 32>;
    __shared__ __attribute__((aligned(16))) float smem[2 * Core::SLOT];
    const int tiles = p.MT * p.NT, split = blockIdx.x / tiles;
    int mt, nt;
    tile_coords(blockIdx.x - split * tiles, p.MT, p.NT, mt, nt);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int nk = p.d / 16, per = (nk + p.splits - 1) / p.splits, k0 = split * per;
    Core core;
    core.a.setup(p.x, p.x, p.d, mt * 64, p.T, p.d, p.d, tid);
    core.b.setup(p.wg, p.wu, p.d, nt * 128, p.F, p.d, p.d, tid);
    f32x16 acc[2];
    core.run(k0, k0 + per < nk ? k0 + per : nk, smem, tid, acc);
    const int n = nt * 64 + (wave & 1) * 32 + (lane & 31);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int m = mt * 64 + (wave >> 1) * 32 + acc_row(i, lane);
        if (m < p.T && n < p.F) {
            const int64_t o = (int64_t)m * p.F + n;
            const float g = acc[0][i], u = acc[1][i];
            if (p.splits > 1) {
                const int64_t part = (int64_t)p.T * p.F;
                p.part[2 * split * part + o] = g;
                p.part[(2 * split + 1) * part + o] = u;
                continue;
            }
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

// The workgroup tiles of the products, and what one stage of 64 K elements and the
// rest of a tile cost on a CU (us, measured on products of many sizes with
// `per_cu` tiles per CU): larger tiles move fewer bytes per product, smaller ones give every
// CU work.  Splitting K does too; the parts are written and read once more.
struct MulTile {
    int bm, bn, per_cu;
    double stage;
};
constexpr MulTile MUL_TILES[] = {{256, 256, 1, 1.5}, {256, 128, 1, 0.88}, {128, 128, 1, 0.52}, {128, 64, 1, 0.36}};
constexpr MulTile MUL_TILE_F32 = {64, 128, 2, 2.9};  // two on a CU
constexpr double MUL_TILE_US = 5, MUL_JOIN_US = 4, MUL_PART_BYTES_PER_US = 4e6;
constexpr int CUS = 256, MUL_MOST_SPLITS = 16;

struct MulPlan {
    int tile, splits;
};

// The tile and the number of K splits with the least estimated time.
static MulPlan mul_plan(const MulTile *tile, int tiles, int64_t M, int64_t N, int64_t K)
{
    MulPlan best{0, 1};
    double best_us = 1e300;
    const int64_t stages = ceil_div(K, 64);
    for (int t = 0; t < tiles; ++t)
        for (int splits = 1; splits <= MUL_MOST_SPLITS && (splits == 1 || splits <= stages); splits *= 2) {
            const int64_t wgs = ceil_div(M, tile[t].bm) * ceil_div(N, tile[t].bn) * splits;
            double us = (double)ceil_div(wgs, CUS * tile[t].per_cu) * ((double)ceil_div(stages, splits) * tile[t].stage + MUL_TILE_US);
            if (splits > 1)
                us += MUL_JOIN_US + (double)M * N * 8 * splits / MUL_PART_BYTES_PER_US;
            if (us < best_us) {
                best_us = us;
                best = MulPlan{t, splits};
            }
        }
    return best;
}

static MulPlan forward_plan(int vdtype, int T, int d, int F)
{
    if (T <= GLU_FEW)
        return {0, 1};
    return vdtype == 1 ? mul_plan(MUL_TILES, 4, T, 2 * (int64_t)F, d) : mul_plan(&MUL_TILE_F32, 1, T, 2 * (int64_t)F, d);
}

size_t glu_forward_ws(int T, int d, int F, int vdtype)
{
    const int splits = forward_plan(vdtype, T, d, F).splits;
    return splits > 1 ? (size_t)splits * 2 * T * F * sizeof(float) : 0;
}

static dim3 join_grid(int64_t n)
{
    const int64_t wgs = ceil_div(n / 4, 256);
    return dim3((unsigned)(wgs < 4096 ? wgs : 4096));
}

hipError_t launch_glu(int vdtype, const GluFwd &args, hipStream_t s)
{
    GluFwd p = args;
    if (p.T <= GLU_FEW) {
        const dim3 grid(p.F / 16), block(256);
        if (vdtype == 1 && p.T <= 32)
            glu_stream_kernel<__bf16, 32, 16, 9><<<grid, block, 0, s>>>(p);
        else if (vdtype == 1)
            glu_stream_kernel<__bf16, 64, 16, 6><<<grid, block, 0, s>>>(p);
        else if (p.T <= 32)
            glu_stream_kernel<float, 32, 16, 9><<<grid, block, 0, s>>>(p);
        else
            glu_stream_kernel<float, 64, 16, 6><<<grid, block, 0, s>>>(p);
        return hipGetLastError();
    }
    const MulPlan plan = forward_plan(vdtype, p.T, p.d, p.F);
    p.splits = plan.splits;
    if (vdtype == 0) {
        p.MT = (int)ceil_div(p.T, 64);
        p.NT = (int)ceil_div(p.F, 64);
        glu_f32_kernel<<<dim3(p.MT * p.NT * p.splits), dim3(256), 0, s>>>(p);
    } else {
        const MulTile &tile = MUL_TILES[plan.tile];
        p.tiles = dg_tiles(ceil_div(p.T, tile.bm), ceil_div(p.F, tile.bn / 2), p.splits);
        const dim3 grid((unsigned)dg_grid(p.tiles));
        switch (plan.tile) {
        case 0:
            glu_kernel<256, 256, 64, 128, 2><<<grid, dim3(512), 0, s>>>(p);
            break;
        case 1:
            glu_kernel<256, 128, 64, 64, 3><<<grid, dim3(512), 0, s>>>(p);
            break;
        case 2:
            glu_kernel<128, 128, 32, 64, 4><<<grid, dim3(512), 0, s>>>(p);
            break;
        default:
            glu_kernel<128, 64, 32, 64, 3><<<grid, dim3(256), 0, s>>>(p);
            break;
        }
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1)
        return e;
    if (vdtype == 1)
        glu_join_act_kernel<__bf16><<<join_grid((int64_t)p.T * p.F), dim3(256), 0, s>>>(p);
    else
        glu_join_act_kernel<float><<<join_grid((int64_t)p.T * p.F), dim3(256), 0, s>>>(p);
    return hipGetLastError();
}

// Tiles and splits of a product of the backward pass.
static MulPlan backward_plan(int vdtype, int64_t M, int64_t N, int64_t K)
{
    if (M == 0 || N == 0 || K == 0)
        return {0, 1};
    return vdtype == 1 ? mul_plan(MUL_TILES, 3, M, N, K) : mul_plan(&MUL_TILE_F32, 1, M, N, K);
}

static size_t up256_(size_t b) { return (b + 255) & ~(size_t)255; }

GluWs glu_backward_ws(int T, int d, int F, int vdtype)
{
    GluWs w{};
    const size_t es = vdtype == 1 ? 2 : 4;
    w.part = up256_((size_t)ceil_div(T, 64) * 64 * glu_pitch(F) * es);
    const MulPlan dx = backward_plan(vdtype, T, d, 2 * (int64_t)F), dw = backward_plan(vdtype, 2 * (int64_t)F, d, T);
    const size_t a = dx.splits > 1 ? (size_t)dx.splits * T * d * 4 : 0;
    const size_t b = dw.splits > 1 ? (size_t)dw.splits * 2 * F * d * 4 : 0;
    w.bytes = w.part + (a > b ? a : b);
    return w;
}

template <bool A_KC, bool B_KC> static hipError_t mul_go(int vdtype, GluMul p, hipStream_t s)
{
    const MulPlan plan = backward_plan(vdtype, p.M, p.N, p.K);
    p.splits = plan.splits;
    if (vdtype == 0) {
        p.MT = (int)ceil_div(p.M, 64);
        p.NT = (int)ceil_div(p.N, 128);
        glu_mul_f32_kernel<A_KC, B_KC><<<dim3(p.MT * p.NT * p.splits), dim3(256), 0, s>>>(p);
    } else {
        const MulTile &tile = MUL_TILES[plan.tile];
        p.tiles = dg_tiles(ceil_div(p.M, tile.bm), ceil_div(p.N, tile.bn), p.splits);
        const dim3 grid((unsigned)dg_grid(p.tiles));
        if (plan.tile == 0)
            glu_mul_kernel<256, 256, 64, 128, 2, A_KC, B_KC><<<grid, dim3(512), 0, s>>>(p);
        else if (plan.tile == 1)
            glu_mul_kernel<256, 128, 64, 64, 3, A_KC, B_KC><<<grid, dim3(512), 0, s>>>(p);
        else
            glu_mul_kernel<128, 128, 32, 64, 4, A_KC, B_KC><<<grid, dim3(512), 0, s>>>(p);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1)
        return e;
    const dim3 join = join_grid((int64_t)p.M * p.N);
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
        const bool once = 3 * (int64_t)p.T * p.F * es > ((int64_t)256 << 20);
        if (vdtype == 1 && once)
            glu_dact_kernel<__bf16, true><<<grid, dim3(256), 0, s>>>(p, rows);
        else if (vdtype == 1)
            glu_dact_kernel<__bf16, false><<<grid, dim3(256), 0, s>>>(p, rows);
        else
            glu_dact_kernel<float, false><<<grid, dim3(256), 0, s>>>(p, rows);
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
