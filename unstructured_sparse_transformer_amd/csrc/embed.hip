// embed.hip -- rows of a table for token ids (twell_embed_forward) and the
// table's gradient (twell_embed_backward).
//
//   out[t] = scale * table[ids[t]]
//   dtable[v] = [old +] scale * sum over the tokens t with ids[t] = v of dout[t]
// A token whose id is none of 0 .. V-1 gets zeros and adds to no row.
//
// Both are bound by memory.  The gradient's sums run in the order of t: the
// tokens are sorted by id first (stable), so that a row of the table is summed by
// one thread per piece of columns, without float atomics.
#include "embed.h"
#include "rows.h"

#include <type_traits>

namespace twell {

// Work item i of a launch's n: rows of `pieces` pieces each, one after another.  A
// workgroup's first row is found once, in 64 bits; its threads count on from there.
struct EmbItem {
    int64_t row;
    int piece;
};
__device__ __forceinline__ EmbItem emb_item(int64_t first, int add, int pieces)
{
    const int64_t row = first / pieces;
    const uint32_t r = (uint32_t)(first - row * pieces) + (uint32_t)add;
    const uint32_t up = r / (uint32_t)pieces;
    return EmbItem{row + up, (int)(r - up * (uint32_t)pieces)};
}

// ------------------------------------------------------------------ forward
// EMB_U items a thread, whose ids and rows are loaded together.  8192 rows of 2048,
// bf16 to fp32: 16 us (5.2 TB/s), 19 us where each call's table is another.
constexpr int EMB_U = 4;

template <typename ID, typename TT, typename TO, int E> __global__ __launch_bounds__(256) void embed_kernel(EmbArgs p)
{
    const int pieces = (p.d + E - 1) / E;
    const int64_t first = (int64_t)blockIdx.x * (256 * EMB_U);
    EmbItem it[EMB_U];
    int key[EMB_U];
#pragma unroll
    for (int u = 0; u < EMB_U; ++u) {
        it[u] = emb_item(first, u * 256 + threadIdx.x, pieces);
        key[u] = it[u].row < p.T ? token_key((const ID *)p.ids, it[u].row, p.V) : p.V;
    }
    RowPiece<TT, E> v[EMB_U];
#pragma unroll
    for (int u = 0; u < EMB_U; ++u)
        if (key[u] < p.V) {
            int from;
            const int c = rows_column<E>(it[u].piece, p.d, from);
            v[u].load((const TT *)p.in + (int64_t)key[u] * p.d + c);
        }
#pragma unroll
    for (int u = 0; u < EMB_U; ++u) {
        if (it[u].row >= p.T)
            continue;
        int from;
        const int c = rows_column<E>(it[u].piece, p.d, from);
        float o[E];
#pragma unroll
        for (int e = 0; e < E; ++e)
            o[e] = key[u] < p.V ? v[u].at(e) * p.scale : 0.f;
        rows_store<E>((TO *)p.out + it[u].row * p.d + c, o, from);
    }
}

// ------------------------------------------------------------------ sorting
// Zeros for the table's gradient, from workgroups behind those that sort: they
// take the time that the sorting leaves the memory idle.  8 KB each, past the caches:
// 1.07 GB in 163 us (6.6 TB/s; 2048 workgroups in strides 233 us).
__device__ __forceinline__ void emb_fill(const EmbArgs &p, int wg, int wgs)
{
    const int64_t bytes = (int64_t)p.V * p.d * (p.bf16_table ? 2 : 4);
    char *at = (char *)p.out, *end = at + bytes;
    char *a = (char *)(((uintptr_t)at + 15) & ~(uintptr_t)15);
    char *z = (char *)((uintptr_t)end & ~(uintptr_t)15);
    if (a > z)
        a = z = end;  // (fewer than 16 bytes)
    if (wg == 0) {
        for (char *q = at + threadIdx.x * 2; q < a && q < end; q += blockDim.x * 2)
            *(uint16_t *)q = 0;
        for (char *q = z + threadIdx.x * 2; q < end; q += blockDim.x * 2)
            *(uint16_t *)q = 0;
    }
    const int64_t n = (z - a) / 16;
    const int64_t per = (n + wgs - 1) / wgs, stop = (wg + 1) * per < n ? (wg + 1) * per : n;
    for (int64_t i = wg * per + threadIdx.x; i < stop; i += blockDim.x)
        __builtin_nontemporal_store(u32x4{0, 0, 0, 0}, reinterpret_cast<u32x4 *>(a) + i);
}

// Up to EMB_FEW tokens in one launch: a token's place is the number of tokens
// with a smaller key, or the same key and an earlier row.  A workgroup takes 16
// tokens, 16 threads each, which compare with every key from LDS (two operations
// a key).  By itself, without zeros, 4 us at 1003 tokens, 7.7 at 4000, 14 at 8192
// (32 tokens of 8 threads leave half of the CUs idle at 4000, 10.5 us).
constexpr int EMB_RANKS = 16, EMB_RANK_SLICES = 256 / EMB_RANKS;
template <typename ID> __global__ __launch_bounds__(256) void emb_rank_kernel(EmbArgs p, int wgs)
{
    __shared__ __attribute__((aligned(16))) int keys[EMB_FEW];
    __shared__ int count[EMB_RANK_SLICES][EMB_RANKS];
    if ((int)blockIdx.x >= wgs) {
        emb_fill(p, (int)blockIdx.x - wgs, (int)gridDim.x - wgs);
        return;
    }
    const int tid = threadIdx.x, groups = (p.T + EMB_RANKS - 1) / EMB_RANKS;
    for (int t0 = 0; t0 < groups * EMB_RANKS; t0 += 256 * 8) {
        int k[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int t = t0 + i * 256 + tid;
            k[i] = token_key((const ID *)p.ids, t < p.T ? t : p.T - 1, p.V);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int t = t0 + i * 256 + tid;
            if (t < groups * EMB_RANKS)
                keys[t] = t < p.T ? k[i] : 0x7FFFFFF0;  // (above V)
        }
    }
    __syncthreads();
    const int own = (int)blockIdx.x, mine = tid % EMB_RANKS, key = keys[own * EMB_RANKS + mine];
    int n = 0;
#pragma unroll 2
    for (int g = tid / EMB_RANKS; g < groups; g += EMB_RANK_SLICES) {
        const int4 *q = reinterpret_cast<const int4 *>(keys + g * EMB_RANKS);
        if (g != own) {
            const int below = key + (g < own);  // of the tokens before, those with the same key count
#pragma unroll
            for (int j = 0; j < EMB_RANKS / 4; ++j) {
                const int4 k = q[j];
                n += k.x < below;
                n += k.y < below;
                n += k.z < below;
                n += k.w < below;
            }
        } else {
            for (int j = 0; j < EMB_RANKS; ++j)
                n += keys[g * EMB_RANKS + j] < key + (j < mine);
        }
    }
    count[tid / EMB_RANKS][mine] = n;
    __syncthreads();
    if (tid < EMB_RANKS && own * EMB_RANKS + tid < p.T) {
        int at = 0;
#pragma unroll
        for (int s = 0; s < EMB_RANK_SLICES; ++s)
            at += count[s][tid];
        p.key[at] = keys[own * EMB_RANKS + tid];
        p.perm[at] = own * EMB_RANKS + tid;
    }
}

// More tokens: passes over digits of the key, least significant first, each a
// count of every workgroup's digits and a stable move (3 and 8 us at 45000 tokens:
// trips to memory one after another).  A workgroup takes `per` (a multiple of 512)
// consecutive tokens.
constexpr int EMB_BINS = 1 << EMB_DIGIT_BITS, EMB_SORT_THREADS = 512;
static_assert(EMB_BINS == EMB_SORT_THREADS, "a thread a digit");

struct EmbPass {
    const int32_t *key, *perm;  // NULL: the ids, in their order
    int32_t *key_out, *perm_out;
    int shift, mask, per, blocks;
};

template <typename ID> __device__ __forceinline__ int emb_key(const EmbArgs &p, const EmbPass &q, int64_t i)
{
    return q.key ? q.key[i] : token_key((const ID *)p.ids, i, p.V);
}

template <typename ID>
__global__ __launch_bounds__(EMB_SORT_THREADS) void emb_count_kernel(EmbArgs p, EmbPass q)
{
    __shared__ int hist[EMB_BINS];
    if ((int)blockIdx.x >= q.blocks) {
        emb_fill(p, (int)blockIdx.x - q.blocks, (int)gridDim.x - q.blocks);
        return;
    }
    const int tid = threadIdx.x;
    hist[tid] = 0;
    __syncthreads();
    const int64_t first = (int64_t)blockIdx.x * q.per, end = first + q.per < p.T ? first + q.per : p.T;
    for (int64_t i = first + tid; i < end; i += EMB_SORT_THREADS)
        atomicAdd(&hist[(emb_key<ID>(p, q, i) >> q.shift) & q.mask], 1);
    __syncthreads();
    p.counts[blockIdx.x * EMB_BINS + tid] = hist[tid];
}

template <typename ID>
__global__ __launch_bounds__(EMB_SORT_THREADS) void emb_move_kernel(EmbArgs p, EmbPass q)
{
    constexpr int NW = EMB_SORT_THREADS / 64;
    __shared__ int at[NW][EMB_BINS];
    __shared__ int sums[NW];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, own = blockIdx.x;
    // this thread's digit: tokens with it in all workgroups, and in those before this one
    int total = 0, before = 0;
    for (int b0 = 0; b0 < q.blocks; b0 += 16) {  // (16 loads at once: one by one 60 us at 45000 tokens)
        int c[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
            c[i] = p.counts[(b0 + i < q.blocks ? b0 + i : 0) * EMB_BINS + tid];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            total += b0 + i < q.blocks ? c[i] : 0;
            before += b0 + i < own ? c[i] : 0;
        }
    }
    int scan = total;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(scan, o, 64);
        scan += lane >= o ? v : 0;
    }
    if (lane == 63)
        sums[wave] = scan;
    __syncthreads();
    int base = scan - total + before;
    for (int w = 0; w < wave; ++w)
        base += sums[w];
    const int64_t first = (int64_t)own * q.per, end = first + q.per < p.T ? first + q.per : p.T;
    for (int64_t i0 = first; i0 < end; i0 += EMB_SORT_THREADS) {
#pragma unroll
        for (int w = 0; w < NW; ++w)
            at[w][tid] = 0;
        __syncthreads();
        const int64_t i = i0 + tid;
        const bool on = i < end;
        const int key = on ? emb_key<ID>(p, q, i) : 0;
        const int digit = (key >> q.shift) & q.mask;
        // the wave's lanes with the same digit
        uint64_t same = __ballot(on);
        for (int b = 0; b < EMB_DIGIT_BITS; ++b) {
            const uint64_t set = __ballot((digit >> b) & 1);
            same &= (digit >> b) & 1 ? set : ~set;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1));
        if (on && rank == 0)
            at[wave][digit] = __popcll(same);
        __syncthreads();
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const int c = at[w][tid];
            at[w][tid] = base;
            base += c;
        }
        __syncthreads();
        if (on) {
            const int to = at[wave][digit] + rank;
            q.key_out[to] = key;
            q.perm_out[to] = q.perm ? q.perm[i] : (int)i;
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------ sums
// The table's row of a sum, or the sum and what was there.
template <typename TT, int E, bool ADD>
__device__ __forceinline__ void emb_write(const EmbArgs &p, int key, int c, int from, const float (&sum)[E],
                                          const RowPiece<TT, E> &old)
{
    float v[E];
#pragma unroll
    for (int e = 0; e < E; ++e)
        v[e] = ADD ? fmaf(sum[e], p.scale, old.at(e)) : sum[e] * p.scale;
    // (without ADD the columns that two pieces have get the same values from both)
    rows_store<E>((TT *)p.out + (int64_t)key * p.d + c, v, ADD ? from : 0);
}

// A run (the sorted tokens of one id) is cut at multiples of the window W.  A wave
// takes a window and 64 pieces of columns: its keys come in one load, its rows (and
// with ADD the table's, of the runs that end) in batches of 8 one batch ahead,
// however its runs lie, and the runs are added up in order.  (All 32 rows at once in
// unrolled code: its instructions arrive later than the rows, 15 us at 1003 tokens
// of 1001 columns; loads and sums behind branches 17 us.)  Few tokens have windows
// of 8: four times the waves, and one batch each.  The sums of cut runs go to `part`: a window's first rows, if the
// run began before it, to its slot 0, its last ones, if the run begins in it and
// goes on, to slot 1.  8192 rows of 2048 fp32 take 19 us, 67 MB read and 33 written.
template <typename TD, typename TT, int E, bool ADD, int W>
__global__ __launch_bounds__(256) void emb_sum_kernel(EmbArgs p, int slices)
{
    constexpr int B = 8;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
    const int w = wave / slices, piece = (wave - w * slices) * 64 + lane, first = w * W;
    if (first >= p.T)
        return;
    // lane l < 32: token l of the window; lane 32: the key after the window, 33: the one before
    const int at = lane <= W ? first + lane : first - 1;
    const bool there = at >= 0 && at < p.T;
    const int keys = there ? p.key[at] : p.V, rows = there && lane < W ? p.perm[at] : 0;
    const bool on = piece < (p.d + E - 1) / E;
    int from = 0;
    const int c = on ? rows_column<E>(piece, p.d, from) : 0;  // (lanes past the columns read the first ones)
    auto key = [&](int j) { return __builtin_amdgcn_readlane(keys, j); };
    struct Batch {
        RowPiece<TD, E> v[B];
        RowPiece<TT, E> old[ADD ? B : 1];
    };
    auto load = [&](int h, Batch &t) {  // (of any token, also where its row is not wanted: no load waits behind a branch)
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const int j = (h + b) & (W - 1), k = key(j);
            t.v[b].load((const TD *)p.in + (int64_t)__builtin_amdgcn_readlane(rows, j) * p.d + c);
            if constexpr (ADD)
                t.old[b].load((const TT *)p.out + (int64_t)(k < p.V ? k : 0) * p.d + c);
        }
    };
    float *part = p.part + 2 * (int64_t)w * emb_pitch(p.d) + c;
    float sum[E];
#pragma unroll
    for (int e = 0; e < E; ++e)
        sum[e] = 0.f;
    bool cut = key(W + 1) == key(0);  // the run at hand began before the window
    auto add = [&](int h, const Batch &t) {
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const int k = key(h + b);
#pragma unroll
            for (int e = 0; e < E; ++e)
                sum[e] += t.v[b].at(e);
            const bool ends = key(h + b + 1) != k;
            if (ends || h + b + 1 == W) {
                if (k < p.V && on) {
                    if (cut || !ends)
                        rows_store<E>(part + (cut ? 0 : emb_pitch(p.d)), sum, 0);
                    else
                        emb_write<TT, E, ADD>(p, k, c, from, sum, t.old[ADD ? b : 0]);
                }
                cut = false;
#pragma unroll
                for (int e = 0; e < E; ++e)
                    sum[e] = 0.f;
            }
        }
    };
    Batch one, two;
    load(0, one);
    if constexpr (W == B) {
        add(0, one);
    } else {
#pragma clang loop unroll(disable)
        for (int h = 0; h < W && key(h) < p.V; h += 2 * B) {
            load(h + B, two);
            add(h, one);
            load(h + 2 * B, one);
            add(h + B, two);
        }
    }
}

// The cut runs: the sums of a run's windows, added by NW waves, each every NW-th in
// order, whose results are added in order.  Bound by its trips to memory: 4 to 5 us.
template <typename TT, int E, int NW> __global__ __launch_bounds__(NW * 64) void emb_join_kernel(EmbArgs p, int W)
{
    __shared__ float all[NW][E][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int pieces = (p.d + E - 1) / E, piece = blockIdx.y * 64 + lane;
    const int windows = (p.T + W - 1) / W;
    const bool on = piece < pieces;
    int from = 0;
    const int c = on ? rows_column<E>(piece, p.d, from) : 0;
    for (int w = blockIdx.x; w + 1 < windows; w += gridDim.x) {
        const int first = w * W, next = first + W;
        const int key = p.key[next], end = p.key[next - 1], begin = p.key[first], before = p.key[first > 0 ? first - 1 : 0];
        // a run that begins in window w and goes on in the next
        if (key >= p.V || end != key || (begin == key && first > 0 && before == key))
            continue;
        // the first window after it that does not begin with it: 64 at a time, and where the run is longer halving
        int hi = w + 2;
        {
            const int probe = w + 2 + lane;
            const uint64_t other = __ballot(probe >= windows || p.key[(int64_t)(probe < windows ? probe : 0) * W] != key);
            if (other) {
                hi += __builtin_ctzll(other);
            } else {
                int lo = hi + 63;
                hi = windows;
                while (hi - lo > 1) {
                    const int mid = lo + (hi - lo) / 2;
                    if (p.key[mid * W] == key)
                        lo = mid;
                    else
                        hi = mid;
                }
            }
        }
        const int n = hi - w;  // sums: slot 1 of w, then slots 0
        float sum[E];
#pragma unroll
        for (int e = 0; e < E; ++e)
            sum[e] = 0.f;
        if (on) {
#pragma unroll 8
            for (int i = wave; i < n; i += NW) {
                RowPiece<float, E> v;
                v.load(p.part + (2 * (int64_t)(w + i) + (i == 0)) * emb_pitch(p.d) + c);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    sum[e] += v.at(e);
            }
        }
#pragma unroll
        for (int e = 0; e < E; ++e)
            all[wave][e][lane] = sum[e];
        __syncthreads();
        if (wave == 0 && on) {
            for (int k = 1; k < NW && k < n; ++k)
#pragma unroll
                for (int e = 0; e < E; ++e)
                    sum[e] += all[k][e][lane];
            RowPiece<TT, E> old;
            if (p.accumulate) {
                old.load((const TT *)p.out + (int64_t)key * p.d + c);
                emb_write<TT, E, true>(p, key, c, from, sum, old);
            } else {
                emb_write<TT, E, false>(p, key, c, from, sum, old);
            }
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------ few tokens
// Up to EMB_ONE tokens in one launch, without sorting: a workgroup takes a token
// and 64 pieces of columns, and if no earlier token has the same id adds the rows of
// all that do: each of its 4 waves every 4th, 8 at a time, in order, and their sums in
// order.  Without ADD the workgroups behind those write zeros to the rows that no
// token has.  (1003 tokens of 1001: sorting, sums and join take 13.4 us in three
// launches, this one 9.9; 256 tokens 13 and 8.)
template <typename ID, typename TD, typename TT, int E, bool ADD>
__global__ __launch_bounds__(256) void emb_one_kernel(EmbArgs p, int slices, int wgs)
{
    constexpr int B = 8, NW = 4, GROUPS = EMB_ONE / 64, MINE = EMB_ONE / 256;
    __shared__ uint64_t same[GROUPS], there[EMB_FILL_ROWS / 64];
    __shared__ int list[EMB_ONE];
    __shared__ float all[NW][E][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const bool fills = (int)blockIdx.x >= wgs;
    const int t = fills ? 0 : blockIdx.x / slices, piece = (blockIdx.x - t * slices) * 64 + lane;
    const int key = p.T > 0 ? token_key((const ID *)p.ids, t, p.V) : p.V;
    int own[MINE];  // of tokens tid, tid + 256, ...
#pragma unroll
    for (int i = 0; i < MINE; ++i) {
        const int at = i * 256 + tid;
        own[i] = i * 256 < p.T ? token_key((const ID *)p.ids, at < p.T ? at : p.T - 1, p.V) : p.V;
        own[i] = at < p.T ? own[i] : p.V;
    }
    if (fills) {
        const int64_t per = emb_fill_rows(p.d), r0 = ((int64_t)blockIdx.x - wgs) * per;
        const int rows = (int)(r0 + per < p.V ? per : p.V - r0);
        if (tid < EMB_FILL_ROWS / 64)
            there[tid] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < MINE; ++i) {
            const int64_t r = own[i] - r0;
            if (own[i] < p.V && r >= 0 && r < rows)
                atomicOr((unsigned long long *)&there[r >> 6], 1ull << (r & 63));
        }
        __syncthreads();
        const int pieces = (p.d + E - 1) / E;
        const float zero[E] = {};
        for (int i = tid; i < rows * pieces; i += 256) {
            const int row = i / pieces;
            if (there[row >> 6] >> (row & 63) & 1)
                continue;
            int from;
            const int c = rows_column<E>(i - row * pieces, p.d, from);
            rows_store<E>((TT *)p.out + (r0 + row) * p.d + c, zero, 0);
        }
        return;
    }
    if (key >= p.V)
        return;
    int earlier = 0;
#pragma unroll
    for (int i = 0; i < MINE; ++i)
        earlier |= own[i] == key && i * 256 + tid < t;
    if (__syncthreads_or(earlier))
        return;
#pragma unroll
    for (int i = 0; i < MINE; ++i) {
        const uint64_t m = __ballot(own[i] == key);
        if (lane == 0)
            same[i * 4 + wave] = m;  // token i 256 + tid is lane `lane` of group 4 i + wave
    }
    __syncthreads();
    int n = 0;
    for (int g = 0; g < GROUPS && g * 64 < p.T; ++g) {
        const uint64_t m = same[g];
        if (g % 4 == wave && (m >> lane & 1))
            list[n + __popcll(m & ((1ull << lane) - 1))] = g * 64 + lane;
        n += __popcll(m);
    }
    int from = 0;
    const bool on = piece < (p.d + E - 1) / E;
    const int c = on ? rows_column<E>(piece, p.d, from) : 0;  // (lanes past the columns read the first ones)
    RowPiece<TT, E> old;
    if constexpr (ADD)
        old.load((const TT *)p.out + (int64_t)key * p.d + c);
    __syncthreads();
    float sum[E];
#pragma unroll
    for (int e = 0; e < E; ++e)
        sum[e] = 0.f;
    for (int i0 = wave; i0 < n; i0 += NW * B) {
        RowPiece<TD, E> v[B];
#pragma unroll
        for (int b = 0; b < B; ++b)
            v[b].load((const TD *)p.in + (int64_t)list[i0 + b * NW < n ? i0 + b * NW : i0] * p.d + c);
#pragma unroll
        for (int b = 0; b < B; ++b)
            if (i0 + b * NW < n)
#pragma unroll
                for (int e = 0; e < E; ++e)
                    sum[e] += v[b].at(e);
    }
    if (n > 1) {
#pragma unroll
        for (int e = 0; e < E; ++e)
            all[wave][e][lane] = sum[e];
        __syncthreads();
        for (int k = 1; k < NW && k < n; ++k)
#pragma unroll
            for (int e = 0; e < E; ++e)
                sum[e] += all[k][e][lane];
    }
    if (wave == 0 && on)
        emb_write<TT, E, ADD>(p, key, c, from, sum, old);
}

// ------------------------------------------------------------------ host
static int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
static size_t up256_(size_t b) { return (b + 255) & ~(size_t)255; }

size_t emb_layout(EmbArgs &a, void *base)
{
    char *at = (char *)base;
    const size_t list = up256_((size_t)a.T * 4);
    auto take = [&](size_t bytes) {
        char *p = at;
        at += bytes;
        return p;
    };
    a.key = (int32_t *)take(list);
    a.perm = (int32_t *)take(list);
    a.part = (float *)take(up256_((size_t)2 * emb_most_windows(a.T, a.d) * emb_pitch(a.d) * 4));
    if (a.T > EMB_FEW) {
        a.key2 = (int32_t *)take(list);
        a.perm2 = (int32_t *)take(list);
        a.counts = (int32_t *)take((size_t)EMB_MOST_BLOCKS * EMB_BINS * 4);
    }
    return at - (char *)base;
}

template <typename ID, typename TT, typename TO> static hipError_t run_embed(const EmbArgs &p, hipStream_t s)
{
    constexpr int E = std::is_same_v<TT, __bf16> && std::is_same_v<TO, __bf16> ? 8 : 4;
    const int per = p.d >= E ? E : 1;
    const dim3 grid((unsigned)ceil_div((int64_t)p.T * ceil_div(p.d, per), 256 * EMB_U));
    if (per == E)
        embed_kernel<ID, TT, TO, E><<<grid, dim3(256), 0, s>>>(p);
    else
        embed_kernel<ID, TT, TO, 1><<<grid, dim3(256), 0, s>>>(p);
    return hipGetLastError();
}

hipError_t launch_embed(const EmbArgs &p, hipStream_t s)
{
    auto with_id = [&](auto id) {
        using ID = decltype(id);
        if (p.bf16_table)
            return p.bf16_rows ? run_embed<ID, __bf16, __bf16>(p, s) : run_embed<ID, __bf16, float>(p, s);
        return p.bf16_rows ? run_embed<ID, float, __bf16>(p, s) : run_embed<ID, float, float>(p, s);
    };
    return p.id64 ? with_id(int64_t{}) : with_id(int32_t{});
}

template <typename ID> static hipError_t run_sort(EmbArgs &p, hipStream_t s)
{
    const int64_t bytes = (int64_t)p.V * p.d * (p.bf16_table ? 2 : 4);
    const int64_t want = p.accumulate ? 0 : ceil_div(bytes, 256 * 16 * 2);
    const int fill = (int)(want < (1 << 20) ? want : 1 << 20);
    if (p.T <= EMB_FEW) {
        const int wgs = (int)ceil_div(p.T, EMB_RANKS);
        if (wgs + fill > 0)
            emb_rank_kernel<ID><<<dim3(wgs + fill), dim3(256), 0, s>>>(p, wgs);
        return hipGetLastError();
    }
    int bits = 1;
    while (((int64_t)1 << bits) <= p.V)  // keys are 0 .. V
        ++bits;
    const int passes = (int)ceil_div(bits, EMB_DIGIT_BITS), each = (int)ceil_div(bits, passes);
    EmbPass q{};
    q.per = (int)(ceil_div(ceil_div(p.T, EMB_MOST_BLOCKS), EMB_SORT_THREADS) * EMB_SORT_THREADS);
    q.blocks = (int)ceil_div(p.T, q.per);
    q.mask = (1 << each) - 1;
    for (int i = 0; i < passes; ++i) {
        const bool last_side = (passes - 1 - i) % 2 == 0;  // the last pass ends in key and perm
        q.key_out = last_side ? p.key : p.key2;
        q.perm_out = last_side ? p.perm : p.perm2;
        q.shift = i * each;
        emb_count_kernel<ID><<<dim3(q.blocks + (i == 0 ? fill : 0)), dim3(EMB_SORT_THREADS), 0, s>>>(p, q);
        emb_move_kernel<ID><<<dim3(q.blocks), dim3(EMB_SORT_THREADS), 0, s>>>(p, q);
        q.key = q.key_out;
        q.perm = q.perm_out;
    }
    return hipGetLastError();
}

template <typename TD, typename TT, int E, int W> static hipError_t run_sums(const EmbArgs &p, hipStream_t s)
{
    const int64_t windows = ceil_div(p.T, W), slices = ceil_div(ceil_div(p.d, E), 64);
    const dim3 grid((unsigned)ceil_div(windows * slices, 4)), block(256);
    if (p.accumulate)
        emb_sum_kernel<TD, TT, E, true, W><<<grid, block, 0, s>>>(p, (int)slices);
    else
        emb_sum_kernel<TD, TT, E, false, W><<<grid, block, 0, s>>>(p, (int)slices);
    if (windows > 1) {
        const int64_t most = ceil_div(2048, slices), x = windows - 1 < most ? windows - 1 : most;
        const dim3 runs((unsigned)x, (unsigned)slices);
        // (a run has at most all windows: up to 64 for each of 4 waves, 128 of 8; the more waves, the fewer of the
        // workgroups that find no run run at once)
        if (windows <= 256)
            emb_join_kernel<TT, E, 4><<<runs, dim3(256), 0, s>>>(p, W);
        else if (windows <= 1024)
            emb_join_kernel<TT, E, 8><<<runs, dim3(512), 0, s>>>(p, W);
        else
            emb_join_kernel<TT, E, 16><<<runs, dim3(1024), 0, s>>>(p, W);
    }
    return hipGetLastError();
}

static int64_t slices_of(int d) { return ceil_div(ceil_div(d, d >= 4 ? 4 : 1), 64); }

template <typename ID, typename TD, typename TT, int E> static hipError_t run_one(const EmbArgs &p, hipStream_t s)
{
    const int64_t slices = slices_of(p.d), wgs = p.T * slices;
    const int64_t fill = p.accumulate ? 0 : ceil_div(p.V, emb_fill_rows(p.d));
    const dim3 grid((unsigned)(wgs + fill)), block(256);
    if (p.accumulate)
        emb_one_kernel<ID, TD, TT, E, true><<<grid, block, 0, s>>>(p, (int)slices, (int)wgs);
    else
        emb_one_kernel<ID, TD, TT, E, false><<<grid, block, 0, s>>>(p, (int)slices, (int)wgs);
    return hipGetLastError();
}

hipError_t launch_embed_backward(const EmbArgs &args, hipStream_t s)
{
    EmbArgs p = args;
    if (p.T == 0 && p.accumulate)
        return hipSuccess;
    const bool one = p.T <= EMB_ONE && p.T * slices_of(p.d) <= EMB_ONE_WGS &&
                     (p.accumulate || (int64_t)p.V * p.d <= EMB_ONE_TABLE);
    if (!one) {
        const hipError_t e = p.id64 ? run_sort<int64_t>(p, s) : run_sort<int32_t>(p, s);
        if (e != hipSuccess || p.T == 0)
            return e;
    }
    auto with = [&](auto rows, auto table) {
        using TD = decltype(rows);
        using TT = decltype(table);
        if (one && p.d >= 4)
            return p.id64 ? run_one<int64_t, TD, TT, 4>(p, s) : run_one<int32_t, TD, TT, 4>(p, s);
        if (one)
            return p.id64 ? run_one<int64_t, TD, TT, 1>(p, s) : run_one<int32_t, TD, TT, 1>(p, s);
        if (p.d < 4)
            return run_sums<TD, TT, 1, EMB_WINDOW>(p, s);
        return p.T <= emb_short(p.d) ? run_sums<TD, TT, 4, EMB_WINDOW_SHORT>(p, s) : run_sums<TD, TT, 4, EMB_WINDOW>(p, s);
    };
    if (p.bf16_table)
        return p.bf16_rows ? with(__bf16{}, __bf16{}) : with(float{}, __bf16{});
    return p.bf16_rows ? with(__bf16{}, float{}) : with(float{}, float{});
}

}  // namespace twell
