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
// dg and du are rounded to the element type, as the matrix units take them: in
// bf16 the gradients are off by 2.3e-3 of their size, where products rounded once are
// by 1.7e-3; operands of 32 bits would take the fp32 units, a ninth of the rate.
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
// Bound by the matrix units.  bf16, 8192 x 2048 x 8192 with g and u kept: 471 us
// on the same inputs again, 487 us on others (1.13 PFLOP/s); the product by itself takes 420 us at the clock the chip's power
// cap leaves it, the rest is 403 MB of results that leave between the tiles
// (workgroups started up to 13 us apart, so that some store while others
// multiply: no change).  fp32, 1500 x 2048 x 2048: 188 us, 134 of 157 TFLOP/s.
// fp32 tiles are small and several share a CU, hence the waves per SIMD.
template <typename TI, int BM, int BN, int WM, int WN, int S>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64) __attribute__((amdgpu_waves_per_eu(2, sizeof(TI) == 4 ? 4 : 2))) void
glu_kernel(GluFwd p)
{
    constexpr int DB = WN / 2, NB = DB / 32;
    using Core = DgCore<TI, BM, BN, WM, WN, true, true, DB, S>;
    __shared__ __attribute__((aligned(16))) char smem[Core::LDS];
    static_assert(sizeof(TI) == 4 || Core::NW * dg_stage_bytes<NB>() <= Core::LDS, "the stores' staging fits");
    int mt, nt, split;
    if (!dg_tile(p.tiles, blockIdx.x, mt, nt, split))
        return;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    Core core;
    const int64_t ld = (int64_t)p.d * sizeof(TI);
    core.a.setup(p.x, p.x, ld, mt * BM, p.T, p.d, 0, wave, lane);
    core.b.setup(p.wg, p.wu, ld, nt * BN, p.F, p.d, 0, wave, lane);
    f32x16 acc[Core::FM][Core::FN];
    const int nk = p.d / Core::A::SK, per = (nk + p.splits - 1) / p.splits, k0 = split * per;
    core.run(k0, k0 + per < nk ? k0 + per : nk, smem, tid, acc);
    const int m0 = mt * BM + wave / Core::NWN * WM, n0 = nt * (BN / 2) + wave % Core::NWN * DB;
    if (p.splits > 1) {
#pragma unroll
        for (int fm = 0; fm < Core::FM; ++fm)
#pragma unroll
            for (int fn = 0; fn < Core::FN; ++fn)
                dg_store_block<TI>(acc[fm][fn], lane, p.part + (int64_t)(split * 2 + fn / NB) * p.T * p.F, p.F,
                                   m0 + fm * 32, n0 + fn % NB * 32, p.T, p.F);
        return;
    }
    if constexpr (sizeof(TI) == 4) {
#pragma unroll
        for (int fm = 0; fm < Core::FM; ++fm)
#pragma unroll
            for (int fn = 0; fn < NB; ++fn) {
                const int m = m0 + fm * 32, n = n0 + fn * 32;
                const f32x16 &g = acc[fm][fn], &u = acc[fm][fn + NB];
                if (p.g)
                    dg_store_block<TI>(g, lane, (float *)p.g, p.F, m, n, p.T, p.F);
                if (p.u)
                    dg_store_block<TI>(u, lane, (float *)p.u, p.F, m, n, p.T, p.F);
                f32x16 h;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    h[i] = glu_act<false>(g[i], p.act) * u[i];
                dg_store_block<TI>(h, lane, (float *)p.h, p.F, m, n, p.T, p.F);
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
// reading the weights once: 67 MB of the 2B-like layer in 12.7 us at T = 1
// (5.3 TB/s) and 13.4 us at T = 64.  Workgroups start at different stages:
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
            a[f] = DgOperand<TI, 32, true, 1>::fragment(cur, f * 32, wave, lane);
#pragma unroll
        for (int f = 0; f < FN; ++f)
            b[f] = DgOperand<TI, 32, true, 1>::fragment(cur + A_BYTES, f * 32, wave, lane);
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
    DgTiles tiles;
    int wg0, wgs;  // its workgroups of the launch (0: not wanted)
};

// Workgroup wg's tile of one product of the backward pass.
template <typename TI, int BM, int BN, int WM, int WN, int S, bool A_KC>
__device__ __forceinline__ void glu_mul_tile(const GluMul &p, int wg, char *smem)
{
    using Core = DgCore<TI, BM, BN, WM, WN, A_KC, false, 0, S>;
    constexpr int SK = Core::A::SK;
    static_assert(sizeof(TI) == 4 || Core::NW * dg_stage_bytes<Core::FN>() <= Core::LDS, "the stores' staging fits");
    int mt, nt, split;
    if (!dg_tile(p.tiles, wg, mt, nt, split))
        return;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    Core core;
    const int nk = (p.K + SK - 1) / SK, per = (nk + p.splits - 1) / p.splits;
    const int k0 = split * per, k1 = k0 + per < nk ? k0 + per : nk;
    core.a.setup(p.a, p.a, p.lda, mt * BM, p.M, nk * SK, nk, wave, lane);
    core.b.setup(p.b, p.b2, p.ldb, nt * BN, p.N, p.K, p.k_turn / SK, wave, lane);
    f32x16 acc[Core::FM][Core::FN];
    core.run(k0, k1, smem, tid, acc);
    const int m0 = mt * BM + wave / Core::NWN * WM, n0 = nt * BN + wave % Core::NWN * WN;
    if (p.splits > 1) {
#pragma unroll
        for (int fm = 0; fm < Core::FM; ++fm)
#pragma unroll
            for (int fn = 0; fn < Core::FN; ++fn)
                dg_store_block<TI>(acc[fm][fn], lane, p.part + (int64_t)split * p.M * p.N, p.N, m0 + fm * 32, n0 + fn * 32,
                                   p.M, p.N);
        return;
    }
    [[maybe_unused]] char *stage = smem + wave * dg_stage_bytes<Core::FN>();
#pragma unroll
    for (int fm = 0; fm < Core::FM; ++fm) {
        int m = m0 + fm * 32;  // m_turn is a multiple of 64: a block of 32 rows lies on one side
        const bool second = m >= p.m_turn;
        TI *out = (TI *)(second ? p.out2 : p.out);
        const int M = second ? p.M - p.m_turn : p.M < p.m_turn ? p.M : p.m_turn;
        m -= second ? p.m_turn : 0;
        if constexpr (sizeof(TI) == 4) {
#pragma unroll
            for (int fn = 0; fn < Core::FN; ++fn)
                dg_store_block<TI>(acc[fm][fn], lane, out, p.N, m, n0 + fn * 32, M, p.N);
        } else {
            dg_store_rows<Core::FN>(stage, lane, [&](int fn, int i) { return acc[fm][fn][i]; }, out, p.N, m, n0, M, p.N);
        }
    }
}

// dx and dW in one launch: neither fills the GPU by itself where rows are few, and
// a launch costs 3 to 4 us.  Bound by the matrix units: the 2B-like layer's two products take 425 us each
// (1.29 PFLOP/s); fp32, 1500 x 2048 x 2048: about 196 and 190 us, 130 TFLOP/s.
template <typename TI, int BM, int BN, int WM, int WN, int S>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64) __attribute__((amdgpu_waves_per_eu(2, sizeof(TI) == 4 ? 4 : 2))) void
glu_mul_kernel(GluMul dx, GluMul dw)
{
    __shared__ __attribute__((aligned(16))) char smem[DgCore<TI, BM, BN, WM, WN, true, false, 0, S>::LDS];
    const int at = (int)blockIdx.x - dx.wg0;
    if (at >= 0 && at < dx.wgs)
        glu_mul_tile<TI, BM, BN, WM, WN, S, true>(dx, at, smem);
    else
        glu_mul_tile<TI, BM, BN, WM, WN, S, false>(dw, (int)blockIdx.x - dw.wg0, smem);
}

// out = sum over the splits of their parts, in order; 4 columns a thread.
template <typename TI> __device__ __forceinline__ void glu_join(const GluMul &p)
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
template <typename TI> __global__ __launch_bounds__(256) void glu_join_kernel(GluMul dx, GluMul dw)
{
    if (dx.wgs > 0 && dx.splits > 1)
        glu_join<TI>(dx);
    if (dw.wgs > 0 && dw.splits > 1)
        glu_join<TI>(dw);
}

// ------------------------------------------------------------------ host
static int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The workgroup tiles of the products, and what they cost (us, measured on
// products of many sizes): `stage` 64 K elements of a tile and `rest` the tile's
// beginning and end, where every CU has its share of the tiles, and a tile that
// has a CU to itself takes `alone` times that.  Larger tiles move fewer bytes per
// product, smaller ones give every CU work.  Splitting K does too; the parts are
// written and read once more.  The constants are a fit to 78 products of 65 to 8192
// rows with every tile and 1 to 8 splits each; the choice is within 1% of the
// best of those on average, and at most 21% (3 us) off.
// bf16: a tile fills a CU.  fp32: 2 to 4 tiles run on one, the matrix unit alone
// sets the time (157 TFLOP/s), and what matters is that no CU is left with one
// tile more than the others: 1500 x 2048 x 2048 forward takes 188 us in tiles of
// 64 x 128 (134 TFLOP/s) and 243 us in 128 x 128, 2000 x 512 x 4096 137 and 132;
// dx of the first 203 us in 64 x 64 and 260 us in 128 x 128, dW 210 and 196.
struct MulTile {
    int bm, bn;
    double stage, rest, alone;
};
constexpr MulTile MUL_TILES[] = {{256, 256, 1.5, 4, 1}, {256, 128, 0.8, 5.5, 1}, {128, 128, 0.6, 5, 1}, {128, 64, 0.41, 6, 1}};
constexpr MulTile FWD_TILES_F32[] = {{128, 128, 3.7, 4, 1.05}, {64, 128, 1.9, 2, 1.1}};
constexpr MulTile MUL_TILES_F32[] = {{128, 128, 3.8, 4, 1.05}, {64, 64, 1.0, 1.5, 1.3}};
constexpr double MUL_JOIN_US = 4, MUL_SPLIT_US = 0.45, MUL_PART_BYTES_PER_US = 5e6;
constexpr int CUS = 256, MUL_MOST_SPLITS = 16;

// The tile and the number of K splits with the least estimated time.
static MulPlan mul_plan(const MulTile *tile, int tiles, int64_t M, int64_t N, int64_t K)
{
    MulPlan best{0, 1};
    double best_us = 1e300;
    const int64_t stages = ceil_div(K, 64);
    for (int t = 0; t < tiles; ++t)
        for (int splits = 1; splits <= MUL_MOST_SPLITS && (splits == 1 || splits <= stages); splits *= 2) {
            const int64_t wgs = ceil_div(M, tile[t].bm) * ceil_div(N, tile[t].bn) * splits;
            double us = (double)ceil_div(ceil_div(wgs, 8), CUS / 8) * ((double)ceil_div(stages, splits) * tile[t].stage + tile[t].rest);
            if (wgs <= CUS)
                us *= tile[t].alone;
            if (splits > 1)
                us += MUL_JOIN_US + MUL_SPLIT_US * splits + (double)M * N * 8 * splits / MUL_PART_BYTES_PER_US;
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
    return vdtype == 1 ? mul_plan(MUL_TILES, 4, T, 2 * (int64_t)F, d) : mul_plan(FWD_TILES_F32, 2, T, 2 * (int64_t)F, d);
}

// The most bytes that a call with up to T rows needs; need(t) is a call's with t
// rows: its plan and its bytes.  Inside 64 rows that fill the same tiles every
// plan's estimate is linear in t (the parts' bytes): a plan that is the cheapest at
// both ends of a range is so throughout, and needs the most at the range's end.
// (18 us of the host at T = 8192, 2048 x 8192, for the backward pass 140.)
template <typename N> static size_t most_bytes(int lo, const N &need, int hi, decltype(need(0)) first, decltype(need(0)) last)
{
    const size_t most = first.bytes > last.bytes ? first.bytes : last.bytes;
    if (hi - lo <= 1 || first.plan == last.plan)
        return most;
    const int mid = lo + (hi - lo) / 2;
    const auto at = need(mid);
    const size_t l = most_bytes(lo, need, mid, first, at), r = most_bytes(mid, need, hi, at, last);
    return l > r ? l : r;
}
template <typename N> static size_t most_bytes_to(int T, const N &need)
{
    size_t most = 0;
    for (int lo = (T - 1) / 64 * 64 + 1; lo > 0 && T > 0; lo -= 64) {
        const int hi = T - lo < 63 ? T : lo + 63;
        const size_t n = most_bytes(lo, need, hi, need(lo), need(hi));
        most = n > most ? n : most;
    }
    return most;
}

static size_t forward_bytes(const MulPlan &plan, int T, int F)
{
    return plan.splits > 1 ? (size_t)plan.splits * 2 * T * F * sizeof(float) : 0;
}
size_t glu_forward_ws(int T, int d, int F, int vdtype) { return forward_bytes(forward_plan(vdtype, T, d, F), T, F); }

size_t glu_forward_most_ws(int T, int d, int F, int vdtype)
{
    struct Need {
        MulPlan plan;
        size_t bytes;
    };
    return most_bytes_to(T, [&](int t) {
        const MulPlan plan = forward_plan(vdtype, t, d, F);
        return Need{plan, forward_bytes(plan, t, F)};
    });
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
    const MulTile &tile = (vdtype == 1 ? MUL_TILES : FWD_TILES_F32)[plan.tile];
    p.tiles = dg_tiles(ceil_div(p.T, tile.bm), ceil_div(p.F, tile.bn / 2), p.splits);
    const dim3 grid((unsigned)dg_grid(p.tiles));
    if (vdtype == 0) {
        if (plan.tile == 0)
            glu_kernel<float, 128, 128, 32, 64, 2><<<grid, dim3(512), 0, s>>>(p);
        else
            glu_kernel<float, 64, 128, 32, 64, 2><<<grid, dim3(256), 0, s>>>(p);
    } else {
        switch (plan.tile) {
        case 0:
            glu_kernel<__bf16, 256, 256, 64, 128, 2><<<grid, dim3(512), 0, s>>>(p);
            break;
        case 1:
            glu_kernel<__bf16, 256, 128, 64, 64, 3><<<grid, dim3(512), 0, s>>>(p);
            break;
        case 2:
            glu_kernel<__bf16, 128, 128, 32, 64, 4><<<grid, dim3(512), 0, s>>>(p);
            break;
        default:
            glu_kernel<__bf16, 128, 64, 32, 64, 3><<<grid, dim3(256), 0, s>>>(p);
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

// The backward pass's products: one launch for both, with one tile, in which an
// XCD's CUs take the workgroups of the product with the longer ones first and the
// other's fill what the last round of those leaves; or one each (6202 x 1984 x
// 6272 640 us in two launches, 700 us in one; 4096 x 1024 x 4096 166 and 147, 300
// x 512 x 512 20 and 15).  The tiles and the splits of each with the least estimated time.
constexpr double MUL_LAUNCH_US = 3, MUL_SURE = 0.94;  // closer than that the estimates do not tell

static GluWs backward_plan(int vdtype, int64_t T, int64_t d, int64_t F)
{
    const MulTile *tile = vdtype == 1 ? MUL_TILES : MUL_TILES_F32;
    const int tiles = vdtype == 1 ? 3 : 2, xcd_cus = CUS / 8;
    const int64_t M[2] = {T, 2 * F}, K[2] = {2 * F, T};
    GluWs best{};
    MulPlan alone[2] = {{0, 1}, {0, 1}};
    double best_us = 1e300, alone_us[2] = {1e300, 1e300};
    for (int t = 0; t < tiles; ++t) {
        struct {
            int64_t n;  // workgroups of an XCD
            double us, join;
        } c[2][5];
        int kinds[2];
        for (int w = 0; w < 2; ++w) {
            const int64_t stages = ceil_div(K[w], 64), wgs = ceil_div(M[w], tile[t].bm) * ceil_div(d, tile[t].bn);
            int k = 0;
            for (int splits = 1; splits <= MUL_MOST_SPLITS && (splits == 1 || splits <= stages); splits *= 2, ++k) {
                auto &p = c[w][k];
                p.n = ceil_div(wgs * splits, 8);
                p.us = (double)ceil_div(stages, splits) * tile[t].stage + tile[t].rest;
                p.join = splits == 1 ? 0 : MUL_SPLIT_US * splits + (double)M[w] * d * 8 * splits / MUL_PART_BYTES_PER_US;
                const double us = (double)ceil_div(p.n, xcd_cus) * p.us * (p.n <= xcd_cus ? tile[t].alone : 1) + p.join +
                                  (splits > 1 ? MUL_JOIN_US : 0);
                if (us < alone_us[w]) {
                    alone_us[w] = us;
                    alone[w] = MulPlan{t, splits};
                }
            }
            kinds[w] = k;
        }
        for (int i = 0; i < kinds[0]; ++i)
            for (int j = 0; j < kinds[1]; ++j) {
                const bool dx_first = c[0][i].us >= c[1][j].us;
                const auto &l = dx_first ? c[0][i] : c[1][j], &s = dx_first ? c[1][j] : c[0][i];
                const int64_t over = l.n % xcd_cus, rounds = l.n / xcd_cus + (over > 0);
                const int64_t left = s.n - (over ? (xcd_cus - over) * (int64_t)(l.us / s.us) : 0);
                double us = (double)rounds * l.us + (left > 0 ? (double)ceil_div(left, xcd_cus) * s.us : 0);
                if (l.n + s.n <= xcd_cus)
                    us *= tile[t].alone;
                us += c[0][i].join + c[1][j].join + (i + j > 0 ? MUL_JOIN_US : 0);
                if (us < best_us) {
                    best_us = us;
                    best.dx = best.dw = MulPlan{t, 1 << i};
                    best.dw.splits = 1 << j;
                    best.dx_first = dx_first;
                }
            }
    }
    best.together = best_us <= MUL_SURE * (alone_us[0] + alone_us[1] + MUL_LAUNCH_US);
    if (!best.together) {
        best.dx = alone[0];
        best.dw = alone[1];
    }
    return best;
}

static size_t up256_(size_t b) { return (b + 255) & ~(size_t)255; }

GluWs glu_backward_ws(int T, int d, int F, int vdtype)
{
    GluWs w = backward_plan(vdtype, T, d, F);
    const size_t es = vdtype == 1 ? 2 : 4;
    w.part_dx = up256_((size_t)ceil_div(T, 64) * 64 * glu_pitch(F) * es);
    w.part_dw = w.part_dx + up256_(w.dx.splits > 1 ? (size_t)w.dx.splits * T * d * 4 : 0);
    w.bytes = w.part_dw + (w.dw.splits > 1 ? (size_t)w.dw.splits * 2 * F * d * 4 : 0);
    return w;
}

size_t glu_backward_most_ws(int T, int d, int F, int vdtype)
{
    struct Plan {
        MulPlan dx, dw;
        bool together;
        bool operator==(const Plan &o) const { return dx == o.dx && dw == o.dw && together == o.together; }
    };
    struct Need {
        Plan plan;
        size_t bytes;
    };
    auto need = [&](int t) {
        const GluWs w = glu_backward_ws(t, d, F, vdtype);
        return Need{Plan{w.dx, w.dw, w.together}, w.bytes};
    };
    const size_t none = need(0).bytes, most = most_bytes_to(T, need);
    return most > none ? most : none;
}

// One launch of the products' workgroups (either may have none).
static hipError_t launch_muls(int vdtype, int tile, const GluMul &dx, const GluMul &dw, hipStream_t s)
{
    const dim3 grid(dx.wgs + dw.wgs);
    if (grid.x == 0)
        return hipSuccess;
    if (vdtype == 0) {
        if (tile == 0)
            glu_mul_kernel<float, 128, 128, 32, 64, 2><<<grid, dim3(512), 0, s>>>(dx, dw);
        else
            glu_mul_kernel<float, 64, 64, 32, 32, 3><<<grid, dim3(256), 0, s>>>(dx, dw);
    } else if (tile == 0) {
        glu_mul_kernel<__bf16, 256, 256, 64, 128, 2><<<grid, dim3(512), 0, s>>>(dx, dw);
    } else if (tile == 1) {
        glu_mul_kernel<__bf16, 256, 128, 64, 64, 3><<<grid, dim3(512), 0, s>>>(dx, dw);
    } else {
        glu_mul_kernel<__bf16, 128, 128, 32, 64, 4><<<grid, dim3(512), 0, s>>>(dx, dw);
    }
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
    const GluWs &w = p.ws;
    GluMul dx{};
    dx.a = p.dgu;
    dx.lda = glu_pitch(p.F) * es;
    dx.ldb = (int64_t)p.d * es;
    dx.N = p.d;
    GluMul dw = dx;
    dx.M = p.T;
    dx.K = 2 * p.F;
    dx.b = p.wg;
    dx.b2 = p.wu;
    dx.k_turn = p.F;
    dx.out = dx.out2 = p.dx;
    dx.m_turn = rows;
    dx.splits = w.dx.splits;
    dx.part = (float *)((char *)p.dgu + w.part_dx);
    dw.M = 2 * p.F;
    dw.K = p.T;
    dw.b = dw.b2 = p.x;
    dw.k_turn = 1 << 30;
    dw.out = p.dwg;
    dw.out2 = p.dwu;
    dw.m_turn = p.F;
    dw.splits = w.dw.splits;
    dw.part = (float *)((char *)p.dgu + w.part_dw);
    for (GluMul *m : {&dx, &dw}) {
        if (!m->out || m->M == 0)
            continue;
        const MulTile &tile = (vdtype == 1 ? MUL_TILES : MUL_TILES_F32)[m == &dx ? w.dx.tile : w.dw.tile];
        m->tiles = dg_tiles(ceil_div(m->M, tile.bm), ceil_div(m->N, tile.bn), m->splits);
        m->wgs = (int)dg_grid(m->tiles);
    }
    if (w.together) {
        (w.dx_first ? dw : dx).wg0 = (w.dx_first ? dx : dw).wgs;
        e = launch_muls(vdtype, w.dx.tile, dx, dw, s);
    } else {
        e = launch_muls(vdtype, w.dx.tile, dx, GluMul{}, s);
        if (e == hipSuccess)
            e = launch_muls(vdtype, w.dw.tile, GluMul{}, dw, s);
    }
    const int64_t parts = (dx.wgs > 0 && dx.splits > 1 ? (int64_t)dx.M * dx.N : 0) + (dw.wgs > 0 && dw.splits > 1 ? (int64_t)dw.M * dw.N : 0);
    if (e != hipSuccess || parts == 0)
        return e;
    if (vdtype == 1)
        glu_join_kernel<__bf16><<<join_grid(parts), dim3(256), 0, s>>>(dx, dw);
    else
        glu_join_kernel<float><<<join_grid(parts), dim3(256), 0, s>>>(dx, dw);
    return hipGetLastError();
}

}  // namespace twell
