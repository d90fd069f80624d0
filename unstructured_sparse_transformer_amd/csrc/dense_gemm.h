// dense_gemm.h -- the matrix-product core of the gated product (gfx950).
//
// C[m][n] = sum_k A(m, k) B(k, n) on workgroup tiles of BM x BN, K in stages of
// 64 bf16 or 32 fp32 elements, fp32 accumulators (v_mfma_f32_32x32x16_bf16, or 4
// of v_mfma_f32_32x32x2f32 on a lane's 4 elements).  In bf16 B's
// fragment is the instruction's first operand: a lane then holds 4 consecutive n
// of one m (element i of lane l of a block: n = 8 (i / 4) + 4 (l / 32) + i % 4,
// m = l % 32), which leave as one 8-byte piece of a row.  In fp32 it is A's: a
// lane has one n, and 32 lanes store 128 bytes of a row (16-byte pieces of 32 rows: 4096
// x 64 x 512 forward 14.3 us, 11.7 so; products in parts 1% the other way).
// Each operand is read as it lies in memory:
//   KC  rows of its M (or N) index, K contiguous:   x and W of the forward pass
//   KS  rows of K, its M (or N) index contiguous:   W in dx, x and dg in dW
// A stage of either is 128 bytes per M (or N) index, copied by global->LDS
// instructions of 1 KiB per wave.  KC stages keep 128-byte rows with XORed
// 16-byte chunks (lds_off); KS stages keep the raw rows, their chunks XORed so
// that a transposing LDS read (ds_read_b64_tr_b16) of 4 bf16 rows, or a read of
// one element a lane of 2 fp32 rows, meets every bank once.
#pragma once

#include "twell_device.h"

namespace twell {

// Tiles' 64-bit base addresses with offsets below 2^31 inside a tile: the matrices
// themselves have no size limit.  An offset of DG_NONE is out of the descriptor's
// range, and reads as zeros.
constexpr int DG_NONE = (int)0x80000000u;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t dg_rsrc(const void *base)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, DG_NONE, 0x00020000);
}

// Waits until at most N copies of this wave are in flight, and for its LDS reads.
template <int N> __device__ __forceinline__ void dg_wait()
{
    static_assert(N <= 63, "vmcnt range");
    __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | ((N >> 4) << 14));
}

// Tiles to workgroups.  Workgroup g runs on XCD g % 8, and each XCD has an L2 of
// its own: the tiles of all K splits stand in one row, split after split, a
// split's in stripes of 8 tile columns, a stripe's in bands of `h` tile rows walked
// column by column, and each XCD takes an eighth of that row.  The 32 workgroups an XCD runs at once then form a block
// of 8 x 4 tiles of one split and read 12 operand tiles instead of up to 33
// (1003 x 1024, K = 8192 in 4 splits: 29 us, and 30 us with all splits on every
// XCD), no XCD has a tile more than its share, and at 8192 rows the XCDs walk down
// A together, each with columns of B of its own (8192 x 2048 x 8192 forward between a
// step's other kernels: 535 us, 557 without stripes).
constexpr int DG_STRIPE = 8;
struct DgTiles {
    int MT, NT, splits, h, per;  // per: tiles of an XCD
};

// Tile (mt, nt) and K split of workgroup g.  False: no tile is left for it.
__device__ __forceinline__ bool dg_tile(const DgTiles &t, int g, int &mt, int &nt, int &split)
{
    const int at = (g & 7) * t.per + (g >> 3), tiles = t.MT * t.NT;
    split = at / tiles;
    int r = at - split * tiles;
    const int stripe = r / (t.MT * DG_STRIPE), n0 = stripe * DG_STRIPE;
    const int w = t.NT - n0 < DG_STRIPE ? t.NT - n0 : DG_STRIPE;
    r -= n0 * t.MT;
    const int band = r / (t.h * w), q = r - band * t.h * w;
    const int left = t.MT - band * t.h, h = left < t.h ? left : t.h;
    nt = q / h;
    mt = band * t.h + q - nt * h;
    nt += n0;
    return split < t.splits;
}

// Bands of equal height, up to the height of the block that an XCD runs at once
// (twice as high as wide).
inline DgTiles dg_tiles(int64_t MT, int64_t NT, int splits)
{
    const int64_t per = (MT * NT * splits + 7) / 8;
    int64_t most = 1;
    while (most < 8 && most * most < 2 * per)
        ++most;
    const int64_t bands = (MT + most - 1) / most;
    return DgTiles{(int)MT, (int)NT, splits, (int)((MT + bands - 1) / bands), (int)per};
}
inline int64_t dg_grid(const DgTiles &t) { return (int64_t)8 * t.per; }

// A transposing LDS read.  `restrict` gives the instruction alias information
// of its own: without any, the compiler waits for every global->LDS copy in
// flight before it (vmcnt(0)), which would serialise copies and products.  The
// waits that are due stand in the K loop.
typedef short dg_v4s __attribute__((ext_vector_type(4)));
__device__ __forceinline__ uint2 dg_read_tr(__attribute__((address_space(3))) dg_v4s *__restrict p)
{
    return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(p));
}

// One operand of a workgroup: IDX tile indices, NW waves.  DB > 0 (KC only):
// the tile's rows alternate between two matrices in blocks of DB (row 2 DB q +
// r, r < DB, is column DB q + r of the first, row 2 DB q + DB + r of the second).
template <typename TI, int IDX, bool KC, int NW, int DB = 0> struct DgOperand {
    static constexpr int ES = sizeof(TI), EPC = 16 / ES;
    static constexpr int SK = 128 / ES;              // K elements of a stage
    static constexpr int BYTES = IDX * 128;
    static constexpr int LD = IDX / 8 / NW;          // 1 KiB copies per wave and stage
    static constexpr int RAW = IDX * ES;             // KS: bytes of a raw row
    static constexpr int RPI = KC ? 8 : 1024 / RAW;  // rows per copy
    static_assert(IDX % (8 * NW) == 0, "copies split over the waves");
    static_assert(KC || (RAW >= 256 && RAW <= 1024), "raw rows span whole 256-byte bank windows");
    // the matrix of a copy goes by its number alone, or by its wave alone
    static constexpr bool BY_COPY = DB > 0 && DB % (8 * NW) == 0;
    static_assert(DB == 0 || (KC && (BY_COPY || 8 * NW % (2 * DB) == 0)), "a copy's rows belong to one matrix");

    const char *ptr;  // at the workgroup's first index and the present stage
    int64_t other;    // bytes from there to the same place of the second matrix (DB; KS: added at stage `turn`)
    int64_t step;     // bytes from one stage to the next
    int turn, last;   // KS: first stage of the second matrix, last stage of all
    int voff[LD], vlast[LD];

    __device__ __forceinline__ static int raw_slot(int r, int c) { return c ^ (ES == 2 ? (r & 3) << 2 : (r & 4) << 1); }

    // idx0: the workgroup's first index, n: indices there are, ld: bytes between rows, k: K elements there are (KS:
    // the last stage's rows past k are zeros).
    __device__ __forceinline__ void setup(const void *p, const void *p2, int64_t ld, int idx0, int n, int k, int turn_,
                                          int wave, int lane)
    {
        turn = turn_;
        last = (k - 1) / SK;
        if constexpr (KC) {
            const int first = DB > 0 ? idx0 / 2 : idx0;  // DB: idx0 counts the rows of both
            ptr = (const char *)p + (int64_t)first * ld;
            other = (const char *)p2 - (const char *)p;
            if (DB > 0 && !BY_COPY && ((wave * 8 / (DB > 0 ? DB : 1)) & 1))
                ptr += other;
            step = 128;
#pragma unroll
            for (int j = 0; j < LD; ++j) {
                const int r = (j * NW + wave) * 8 + (lane >> 3);
                const int c = (lane & 7) ^ ((r >> 1) & 7);
                constexpr int D = DB > 0 ? DB : 1;
                int q = DB > 0 ? r / (2 * D) * D + r % D : r;
                q = first + q < n ? q : n - 1 - first;  // rows past the end repeat the last; their results are dropped
                voff[j] = q * (int)ld + c * 16;
            }
        } else {
            ptr = (const char *)p + (int64_t)idx0 * ES;
            step = SK * ld;
            other = (const char *)p2 - (const char *)p - turn_ * step;
#pragma unroll
            for (int j = 0; j < LD; ++j) {
                const int r = (j * NW + wave) * RPI + lane / (RAW / 16);
                int c = raw_slot(r, lane % (RAW / 16)) * EPC;
                c = idx0 + c <= n - EPC ? c : n - EPC - idx0;
                voff[j] = r * (int)ld + c * ES;
                vlast[j] = last * SK + r < k ? voff[j] : DG_NONE;
            }
        }
    }

    // Goes from stage 0 to stage kt, or from stage kt - 1 on to stage kt: what
    // changes from stage to stage is done here, once, and not at every copy.
    __device__ __forceinline__ void start(int kt)
    {
        ptr += kt * step + (!KC && kt >= turn ? other : 0);
        tail(kt);
    }
    __device__ __forceinline__ void next(int kt)
    {
        ptr += step;
        if (!KC && kt == turn)
            ptr += other;
        tail(kt);
    }
    __device__ __forceinline__ void tail(int kt)
    {
        if constexpr (!KC) {
            if (kt == last) {
#pragma unroll
                for (int j = 0; j < LD; ++j)
                    voff[j] = vlast[j];
            }
        }
    }

    // Copy j of the present stage into the operand's LDS area.
    __device__ __forceinline__ void copy(int j, char *lds, int wave) const
    {
        constexpr int D = DB > 0 ? DB : 1;
        const bool second = BY_COPY && ((j * NW * 8 / D) & 1);
        dma16(dg_rsrc(second ? ptr + other : ptr), lds + (j * NW + wave) * 1024, voff[j], 0);
    }

    // The fragment of 32 indices from i0, K sub-step ss (16 elements, fp32: 8):
    // lane l holds index i0 + l % 32, elements 16 ss + 8 (l / 32) .. + 7 (fp32:
    // 8 ss + 4 (l / 32) .. + 3).
    __device__ __forceinline__ static u32x4 fragment(const char *lds, int i0, int ss, int lane)
    {
        if constexpr (KC) {
            return *reinterpret_cast<const u32x4 *>(lds + lds_off<128>(i0 + (lane & 31), ss * 2 + (lane >> 5)));
        } else if constexpr (ES == 4) {
            const int r = ss * 8 + ((lane >> 5) << 2), i = i0 + (lane & 31);
            const char *a = lds + r * RAW + (raw_slot(r, i >> 2) << 4) + ((i & 3) << 2);
            u32x4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] = *reinterpret_cast<const uint32_t *>(a + e * RAW);
            return v;
        } else {
            // Within a 16-lane group the transposing read hands lane i element i % 4 of the 8-byte pieces addressed
            // by lanes i / 4 + 4 j (j < 4) as its values j: lane p addresses row k0 + p / 4 (+ 4 for the second
            // half), columns 4 (p % 4) .. + 3 of the group's 16.
            const int grp = lane >> 4, p = lane & 15;
            const int k0 = ss * 16 + ((grp >> 1) << 3) + (p >> 2);
            const int i = i0 + ((grp & 1) << 4) + ((p & 3) << 2);
            uint2 w[2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int r = k0 + 4 * half;
                const char *a = lds + r * RAW + (raw_slot(r, i >> 3) << 4) + (((i >> 2) & 1) << 3);
                w[half] = dg_read_tr((__attribute__((address_space(3))) dg_v4s *)(a));
            }
            return u32x4{w[0].x, w[0].y, w[1].x, w[1].y};
        }
    }
};

// Waves of WM x WN on tiles of BM x BN, S LDS slots of a stage.  256 x 256 tiles
// of 8 waves reach 1.40 PFLOP/s at 8192^3 with both operands KC, 1.29 at 8192 x
// 2048 x 16384 with B KS and 1.30 at 16384 x 2048 x 8192 with both KS.  There the
// chip runs at about 1.7 GHz under its power cap with the MFMA pipes 0.7 busy;
// the same kernels on zeros reach 1.76 PFLOP/s.  4 waves of 128 x 128 (a third
// fewer LDS reads, one wave a SIMD) measured 3-6% slower, 16 waves of 64 x 64 5%,
// v_mfma_f32_16x16x32_bf16 in the place of 32x32x16 4-7%.
template <typename TI, int BM, int BN, int WM, int WN, bool A_KC, bool B_KC, int DB = 0, int S = 2> struct DgCore {
    static constexpr int NWM = BM / WM, NWN = BN / WN, NW = NWM * NWN, THREADS = NW * 64;
    static constexpr int FM = WM / 32, FN = WN / 32;
    using A = DgOperand<TI, BM, A_KC, NW>;
    using B = DgOperand<TI, BN, B_KC, NW, DB>;
    static constexpr int STAGE = A::BYTES + B::BYTES;
    static constexpr int LDS = S * STAGE;  // S slots
    static constexpr int COPIES = A::LD + B::LD;
    static_assert(DB == 0 || WN == 2 * DB, "a wave holds both products of its columns");

    A a;
    B b;

    __device__ __forceinline__ void copy(int c, char *buf, int wave) const
    {
        if (c < A::LD)
            a.copy(c, buf, wave);
        else
            b.copy(c - A::LD, buf + A::BYTES, wave);
    }
    __device__ __forceinline__ void next(int kt)
    {
        a.next(kt);
        b.next(kt);
    }

    // One sub-step: the MFMAs of fragments af, bf, and between them, in this
    // order, the reads of the next sub-step's fragments (one before each of the
    // first MFMAs) and copies C0..C1-1 of the operands' present stage.  Spread like this neither
    // queue fills up and the MFMA pipe is not held by either (all reads first
    // cost 2-4% of a large product).  The order of the products changes one
    // fragment at a time: fewer operand bits toggle, and the power that is drawn
    // sets the clock (0.5%).
    template <int C0, int C1>
    __device__ __forceinline__ void step(const char *rbuf, int rss, u32x4 (&an)[FM], u32x4 (&bn)[FN],
                                         const u32x4 (&af)[FM], const u32x4 (&bf)[FN], f32x16 (&acc)[FM][FN], int wm,
                                         int wn, int lane, char *cbuf, int wave, bool on) const
    {
        constexpr int NM = FM * FN, NC = C1 - C0, NR = FM + FN;
#pragma unroll
        for (int q = 0; q < NM; ++q) {
#pragma unroll
            for (int r = 0; r < NR; ++r)
                if ((NR <= NM ? r : r * NM / NR) == q) {
                    if (r == 0)
                        bn[0] = B::fragment(rbuf + A::BYTES, wn * WN, rss, lane);
                    else if (r <= FM)
                        an[r - 1] = A::fragment(rbuf, wm * WM + (r - 1) * 32, rss, lane);
                    else
                        bn[r - FM] = B::fragment(rbuf + A::BYTES, wn * WN + (r - FM) * 32, rss, lane);
                }
            __builtin_amdgcn_sched_barrier(0);
            const int fn = q / FM, fm = fn & 1 ? FM - 1 - q % FM : q % FM;
            if constexpr (sizeof(TI) == 4)
                mfma_chunk(TI{}, af[fm], bf[fn], acc[fm][fn]);
            else
                mfma_chunk(TI{}, bf[fn], af[fm], acc[fm][fn]);
#pragma unroll
            for (int c = C0; c < C1; ++c)
                if ((c - C0) * NM / (NC > 0 ? NC : 1) == q && on)
                    copy(c, cbuf, wave);
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // Stages [k0, k1) through S LDS slots: the copies of stage kt + S go into
    // stage kt's slot once the barrier before stage kt's last sub-step has
    // passed, half between that sub-step's MFMAs and half between the next
    // one's, and fragments are read one sub-step ahead.  Ends with a barrier: the
    // caller may use `smem`.
    __device__ __forceinline__ void run(int k0, int k1, char *smem, int tid, f32x16 (&acc)[FM][FN])
    {
        constexpr int H = COPIES / 2;
        const int lane = tid & 63;
        const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int wm = wave / NWN, wn = wave % NWN;
#pragma unroll
        for (int fm = 0; fm < FM; ++fm)
#pragma unroll
            for (int fn = 0; fn < FN; ++fn)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    acc[fm][fn][i] = 0.f;
        if (k0 < k1) {
            a.start(k0);
            b.start(k0);
#pragma unroll
            for (int c = 0; c < COPIES; ++c)
                copy(c, smem, wave);
#pragma unroll
            for (int k = 1; k < S; ++k)
                if (k0 + k < k1) {
                    next(k0 + k);
#pragma unroll
                    for (int c = 0; c < COPIES; ++c)
                        copy(c, smem + k * STAGE, wave);
                }
            if (k0 + S - 1 < k1)
                dg_wait<(S - 1) * COPIES>();
            else
                dg_wait<0>();
            wg_barrier();
            u32x4 af[2][FM], bf[2][FN];
#pragma unroll
            for (int f = 0; f < FM; ++f)
                af[0][f] = A::fragment(smem, wm * WM + f * 32, 0, lane);
#pragma unroll
            for (int f = 0; f < FN; ++f)
                bf[0][f] = B::fragment(smem + A::BYTES, wn * WN + f * 32, 0, lane);
            int slot = 0;
#pragma clang loop unroll(disable)
            for (int kt = k0; kt < k1; ++kt) {
                const int nslot = slot + 1 == S ? 0 : slot + 1, pslot = slot == 0 ? S - 1 : slot - 1;
                char *cur = smem + slot * STAGE, *nxt = smem + nslot * STAGE, *prv = smem + pslot * STAGE;
                const bool pend = kt > k0 && kt - 1 + S < k1;  // the second half of the copies begun in stage kt - 1
                step<H, COPIES>(cur, 1, af[1], bf[1], af[0], bf[0], acc, wm, wn, lane, prv, wave, pend);
                step<0, 0>(cur, 2, af[0], bf[0], af[1], bf[1], acc, wm, wn, lane, nxt, wave, false);
                step<0, 0>(cur, 3, af[1], bf[1], af[0], bf[0], acc, wm, wn, lane, nxt, wave, false);
                __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the slot has been read
                if (kt + 1 < k1) {
                    // stage kt + 1 has arrived; the S - 2 after it may be on their way
                    if (kt + S - 1 < k1)
                        dg_wait<(S - 2) * COPIES>();
                    else
                        dg_wait<0>();
                    wg_barrier();
                }
                if (kt + S < k1)
                    next(kt + S);
                // (after the last stage this reads the other slot as it is; the values are not used)
                step<0, H>(nxt, 0, af[0], bf[0], af[1], bf[1], acc, wm, wn, lane, cur, wave, kt + S < k1);
                slot = nslot;
            }
        }
        __syncthreads();
    }
};

// A block of 32 x 32 accumulators to memory, in fp32.
template <typename TI>
__device__ __forceinline__ void dg_store_block(const f32x16 &v, int lane, float *out, int64_t ld, int m0, int n0, int M, int N)
{
    if constexpr (sizeof(TI) == 4) {
        const int n = n0 + (lane & 31);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int m = m0 + acc_row(i, lane);
            if (m < M && n < N)
                out[m * ld + n] = v[i];
        }
    } else {
        const int m = m0 + (lane & 31);
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const int n = n0 + acc_row(i, lane);
            if (m < M && n < N)
                *reinterpret_cast<float4 *>(out + m * ld + n) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        }
    }
}

// A wave's block of 32 rows by 32 NB columns in bf16, from accumulators
// (value(fn, i)) to memory by way of LDS: 16-byte stores of whole row pieces.
// `lds`: dg_stage_bytes<NB>() bytes of the wave's own.  A row's 16-byte chunks are
// XORed with the row's index among the rows that share a place in the 256-byte
// bank window, and rows 16 on swap a chunk's halves, so that the 32 rows' 8-byte
// pieces of one write, and 16 chunks of one read, meet every bank once.  ONCE:
// not read again soon, written past the caches.
template <int NB> constexpr int dg_stage_bytes() { return 32 * 64 * NB; }
template <int NB> __device__ __forceinline__ int dg_stage_chunk(int row, int chunk)
{
    constexpr int LOG = NB == 4 ? 0 : NB == 2 ? 1 : 2;  // log2(rows per bank window)
    static_assert(NB == 1 || NB == 2 || NB == 4, "rows of 64, 128 or 256 bytes");
    return row * (64 * NB) + ((chunk ^ ((row >> LOG) & (4 * NB - 1))) << 4);
}
template <int NB, bool ONCE = false, typename V>
__device__ __forceinline__ void dg_store_rows(char *lds, int lane, V value, __bf16 *out, int64_t ld, int m0, int n0,
                                              int M, int N)
{
    const int row = lane & 31, half = (lane >> 5) ^ (row >> 4);
    asm volatile("" ::: "memory");
#pragma unroll
    for (int fn = 0; fn < NB; ++fn)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const bf16x2 lo = {(__bf16)value(fn, i), (__bf16)value(fn, i + 1)};
            const bf16x2 hi = {(__bf16)value(fn, i + 2), (__bf16)value(fn, i + 3)};
            *reinterpret_cast<uint2 *>(lds + dg_stage_chunk<NB>(row, fn * 4 + (i >> 2)) + half * 8) =
                make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
        }
    asm volatile("" ::: "memory");
    constexpr int CPR = 4 * NB;  // 16-byte chunks of a row
#pragma unroll
    for (int c0 = 0; c0 < 32 * CPR; c0 += 64) {
        const int r = c0 / CPR + lane / CPR, q = lane % CPR;
        u32x4 v = *reinterpret_cast<const u32x4 *>(lds + dg_stage_chunk<NB>(r, q));
        if (c0 / CPR >= 16)
            v = u32x4{v[2], v[3], v[0], v[1]};
        u32x4 *o = reinterpret_cast<u32x4 *>(out + (int64_t)(m0 + r) * ld + n0 + q * 8);
        if (m0 + r < M && n0 + q * 8 < N) {
            if constexpr (ONCE)
                __builtin_nontemporal_store(v, o);
            else
                *o = v;
        }
    }
    asm volatile("" ::: "memory");
}

}  // namespace twell
