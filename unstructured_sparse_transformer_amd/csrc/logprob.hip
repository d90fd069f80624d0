// logprob.hip -- log probabilities of given tokens from logits, the rows'
// entropy and their most likely tokens (twell_logprob_forward), and the logits'
// gradient (twell_logprob_backward).
//
// A row z of V logits, scaled by c (an inverse temperature), with m = max z:
//   S = sum exp(c (z - m)),  W = sum c (z - m) exp(c (z - m)),  L = log S
//   logp[v] = c (z[v] - m) - L,   entropy H = L - W / S
//   dz[v] = c (dlogp (1[v = target] - p[v]) - dH p[v] (logp[v] + H))
// Everything is relative to m, so nothing of size c m cancels, and H is a sum of two
// terms of one sign.  Below S = 2 one logit is above all others, whose sum would lose
// its digits next to that one's 1: it is taken apart from it (lp_others), so that a
// confident row's L = log(1 + (S - 1)), H and 1 - p are right relative to themselves.
// A row is read once, with the running maximum and sums of each thread (a larger
// maximum scales the sums before it); a logit of -inf has p = 0, and its term of W is
// 0.  Exponentials are in base 2, as the hardware has them.
#include "logprob.h"
#include "rows.h"
#include "wave_ops.h"

#include <type_traits>

namespace twell {

constexpr float LP_LOG2E = 1.44269504088896340736f, LP_LN2 = 0.69314718055994530942f;
constexpr float LP_LEAST = -150.f;  // exp2 of it is 0; in the place of -inf, whose product with 0 is none

// exp2's argument of a logit: (z - m) c, at least LP_LEAST (v_max drops the NaN of -inf - -inf).
__device__ __forceinline__ float lp_arg(float z, float m, float c) { return fmaxf((z - m) * c, LP_LEAST); }
__device__ __forceinline__ float lp_exp2(float x) { return __builtin_amdgcn_exp2f(x); }

// The larger one, or NaN if either is (v_maximum3): a row's maximum tells of a NaN in it.
__device__ __forceinline__ float lp_max(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// What is known of a part of a row: its largest logit, and relative to that the
// sums of exp2(x) and of x exp2(x).
struct LpState {
    float m, s, w;

    // The sums relative to a maximum that is no smaller.
    __device__ __forceinline__ void raise(float to, float c)
    {
        const float by = lp_arg(m, to, c), f = lp_exp2(by);
        w = f * fmaf(s, by, w);
        s *= f;
        m = to;
    }
    __device__ __forceinline__ void join(LpState o, float c)
    {
        const float to = lp_max(m, o.m);
        raise(to, c);
        o.raise(to, c);
        s += o.s;
        w += o.w;
    }
    __device__ __forceinline__ void add(float z, float c)
    {
        const float x = lp_arg(z, m, c), e = lp_exp2(x);
        s += e;
        w = fmaf(x, e, w);
    }
};

// A logit's place in the order of the alternatives: larger values first, then
// lower indices (+0 and -0 are the same value).  0 comes after all of them.
__device__ __forceinline__ uint32_t lp_order(float z)
{
    const uint32_t b = __float_as_uint(z + 0.f);
    return b ^ (b >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ uint64_t lp_key(float z, int v) { return (uint64_t)lp_order(z) << 32 | (0xFFFFFFFFu - (uint32_t)v); }
__device__ __forceinline__ float lp_value(uint32_t order)
{
    return __uint_as_float(order ^ (order >> 31 ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ float lp_key_value(uint64_t key) { return lp_value((uint32_t)(key >> 32)); }
__device__ __forceinline__ int lp_key_index(uint64_t key) { return (int)(0xFFFFFFFFu - (uint32_t)key); }

// The whole sums of a row or of a segment of one: more = S - 1, of nothing but masked
// logits -1.
struct LpSum {
    float m, more, w;
};

// log(1 + y) for y from 0 to 1, right relative to itself within 8 roundings: twice the
// series of artanh at y / (2 + y), at most a third; the first term left out is 2^-26.
// (log1pf has ten times the operations: 16000 x 1404 confident rows 17.6 us with it, 14.2 without.)
__device__ __forceinline__ float lp_log1p(float y)
{
    const float r = y * __builtin_amdgcn_rcpf(2.f + y), q = r * r;
    float t = 1.f / 13.f;
    t = fmaf(t, q, 1.f / 11.f);
    t = fmaf(t, q, 1.f / 9.f);
    t = fmaf(t, q, 1.f / 7.f);
    t = fmaf(t, q, 1.f / 5.f);
    t = fmaf(t, q, 1.f / 3.f);
    return 2.f * fmaf(t * q, r, r);
}

// The value of a row's results from its whole sums.
struct LpRow {
    float m, size2, entropy;  // size2 = log2 S
    bool bad, empty;
    __device__ __forceinline__ LpRow(const LpSum &t) : m(t.m), bad(!(t.m < INFINITY)), empty(t.m == -INFINITY)
    {
        const float s = 1.f + t.more;
        size2 = empty ? 0.f : s < 2.f ? LP_LOG2E * lp_log1p(t.more) : __builtin_amdgcn_logf(s);
        entropy = empty ? 0.f : LP_LN2 * (size2 - t.w / s);
    }
    __device__ __forceinline__ float logp(float z, float scale) const
    {
        if (bad)
            return __uint_as_float(0x7FC00000u);
        return empty ? -INFINITY : (z - m) * scale - LP_LN2 * size2;
    }
};

// A row's results; `given`: its token's logit is z.
__device__ __forceinline__ void lp_finish(const LpArgs &p, int64_t t, const LpSum &sum, bool given, float z)
{
    const LpRow row(sum);
    const float nan = __uint_as_float(0x7FC00000u);
    if (p.norm) {
        p.norm[2 * t] = row.bad ? nan : row.m;
        p.norm[2 * t + 1] = row.bad ? nan : LP_LN2 * row.size2;
    }
    if (p.entropy)
        p.entropy[t] = row.bad ? nan : row.entropy;
    if (p.logp)
        p.logp[t] = given ? row.logp(z, p.scale) : 0.f;
}

constexpr int LP_THREADS = 256, LP_CAND = 1024;
constexpr int LP_MANY = 192;  // logits that reach a bound, from which on equal ones are told apart first
constexpr int LP_SEG = 4096, LP_MOST_SEGS = 64, LP_ONCE = 4;

// Workgroup-wide scratch of the alternatives.
struct LpTop {
    uint32_t tau[LP_THREADS / 64];
    int count, n_threads;
    int cand_threads[LP_THREADS];
    uint64_t cand[LP_CAND];
    uint64_t best[LP_THREADS];
    uint64_t win;
};

// The r-th largest (r from 1 to 64) of the wave's values, bit by bit: the largest
// number that r of them reach.  (Taking the largest out r - 1 times costs as much at
// r = 4, three times as much at 16.)
__device__ __forceinline__ uint32_t lp_nth(uint32_t v, int r)
{
    uint32_t at = 0;
#pragma unroll
    for (int bit = 31; bit >= 0; --bit) {
        const uint32_t up = at | 1u << bit;
        at = __popcll(__ballot(v >= up)) >= r ? up : at;
    }
    return at;
}

// The k best keys of cand[0 .. n), best first, to emit(rank, key).
template <typename F> __device__ __forceinline__ void lp_rank(const uint64_t *cand, int n, int k, int tid, F emit)
{
    for (int i = tid; i < n; i += LP_THREADS) {
        const uint64_t mine = cand[i];
        int above = 0;
#pragma unroll 8
        for (int j = 0; j < n; ++j)
            above += cand[j] > mine;
        if (above < k)
            emit(above, mine);
    }
}

__device__ __forceinline__ void lp_offer(LpTop &sh, float x, int v)
{
    const int at = atomicAdd(&sh.count, 1);
    if (at < LP_CAND)
        sh.cand[at] = lp_key(x, v);
}

// Lists the logits of a segment that reach the order `least`.  The pieces of the few
// threads that have any, a few kilobytes that the caches hold, are read again by all
// (from the registers that they are in: 32 comparisons by every wave, 16000 x 5080
// bf16 109 us in the place of 65), and a lane takes its places in the list at once.
template <typename TI, int E>
__device__ __forceinline__ void lp_list(const TI *z, int v0, int n, uint32_t head, uint32_t least, LpTop &sh, int tid)
{
    const int whole = n / E, rest = n - whole * E, each = (whole + LP_THREADS - 1) / LP_THREADS;
    if (head >= least)
        sh.cand_threads[atomicAdd(&sh.n_threads, 1)] = tid;
    __syncthreads();
    const int nt = sh.n_threads;
    if (nt > LP_MANY) {  // at least so many logits reach it
        if (tid == 0)
            sh.count = nt;
        return;
    }
    for (int i = tid; i < nt * (each + 1); i += LP_THREADS) {
        const int of = sh.cand_threads[i / (each + 1)], j = i % (each + 1);
        if (j < each) {
            const int at = (j * LP_THREADS + of) * E;
            if (at + E > n)
                continue;
            RowPiece<TI, E> x;
            x.load(z + at);
            int hits = 0;
#pragma unroll
            for (int e = 0; e < E; ++e)
                hits += lp_order(x.at(e)) >= least;
            if (hits) {
                int to = atomicAdd(&sh.count, hits);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (lp_order(x.at(e)) >= least) {
                        if (to < LP_CAND)
                            sh.cand[to] = lp_key(x.at(e), v0 + at + e);
                        ++to;
                    }
            }
        } else if (of < rest) {
            const float x = (float)z[whole * E + of];
            if (lp_order(x) >= least)
                lp_offer(sh, x, v0 + whole * E + of);
        }
    }
}

// The k best logits of the segment [v0, v0 + n) of a row, best first, to
// emit(rank, key); emit(rank, 0) where there are fewer.  `largest`: the largest of
// those that this thread has read: pieces tid, tid + 256, ... of E elements, and
// element tid of the rest; own(f) calls f(logit, index) for each of them.  In each
// of the N waves whose threads all have logits, k / N threads have a largest that
// reaches the (k / N)-th largest of the wave's: the lowest of these values is a bound
// that k logits reach (a row too short for one such wave has its first wave's k-th,
// or none).  Only
// threads whose largest reaches it have any that do; the logits that reach it are
// ranked by comparing each with each.  Where many do (equal logits in bulk), those
// above the bound are listed, and then as many of the equal ones as are wanted, the
// lowest indices first.  If even those above the bound are more than the list holds
// (all in few threads), the best is taken k times: a tournament of the threads' best
// remaining.
template <typename TI, int E, typename O, typename F>
__device__ __forceinline__ void lp_alternatives(const TI *z, int v0, int n, int k, float largest, O own, LpTop &sh, int tid, F emit)
{
    const int whole = n / E, rest = n - whole * E, lane = tid & 63, each = (whole + LP_THREADS - 1) / LP_THREADS;
    const uint32_t head = lp_order(largest);
    const int have = whole > rest ? whole : rest, full = have < LP_THREADS ? have / 64 : LP_THREADS / 64;
    uint32_t tau = 0xFFFFFFFFu;
    if ((tid >> 6) < full)
        tau = lp_nth(head, (k + full - 1) / full);
    else if (full == 0 && tid < 64)
        tau = k <= have ? lp_nth(head, k) : lp_order(-INFINITY);
    if (lane == 0)
        sh.tau[tid >> 6] = tau;
    if (tid == 0) {
        sh.count = 0;
        sh.n_threads = 0;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < LP_THREADS / 64; ++w)
        tau = sh.tau[w] < tau ? sh.tau[w] : tau;
    lp_list<TI, E>(z, v0, n, head, tau, sh, tid);
    __syncthreads();
    int found = sh.count;
    if (found > LP_MANY) {
        __syncthreads();
        if (tid == 0)
            sh.count = 0;
        __syncthreads();
        if (head > tau)
            own([&](float x, int v) {
                if (lp_order(x) > tau)
                    lp_offer(sh, x, v);
            });
        __syncthreads();
        found = sh.count;
        // the equal ones in order: the pieces of one round of the threads, then the rest
        for (int j = 0; j <= each && found < k; ++j) {
            const int at = j < each ? (j * LP_THREADS + tid) * E : whole * E + tid, m = j < each ? (at + E <= n ? E : 0) : tid < rest;
            uint32_t same = 0;
            for (int e = 0; e < m; ++e)
                same |= (uint32_t)(lp_order((float)z[at + e]) == tau) << e;
            int total, before = wave_excl_scan(__popc(same), lane, total);
            if (lane == 0)
                sh.tau[tid >> 6] = (uint32_t)total;
            __syncthreads();
            total = 0;
#pragma unroll
            for (int w = 0; w < LP_THREADS / 64; ++w) {
                before += w < tid >> 6 ? (int)sh.tau[w] : 0;
                total += (int)sh.tau[w];
            }
            for (int e = 0, to = found + before; e < m && to < k; ++e)
                if (same >> e & 1)
                    sh.cand[to++] = (uint64_t)tau << 32 | (0xFFFFFFFFu - (uint32_t)(v0 + at + e));
            found = found + total < k ? found + total : k;
            __syncthreads();
        }
    }
    if (found <= LP_CAND) {
        for (int r = tid; r < k; r += LP_THREADS)
            if (r >= found)
                emit(r, (uint64_t)0);
        lp_rank(sh.cand, found, k, tid, emit);
        return;
    }
    // a thread's best key below `under`
    auto best_of = [&](int t, int j0, int step, uint64_t under) {
        uint64_t b = 0;
        auto see = [&](float x, int v) {
            const uint64_t key = lp_key(x, v);
            b = key < under && key > b ? key : b;
        };
        for (int j = j0; j < each; j += step) {
            const int at = (j * LP_THREADS + t) * E;
            if (at + E <= n) {
                RowPiece<TI, E> v;
                v.load(z + at);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    see(v.at(e), v0 + at + e);
            }
        }
        if (j0 == 0 && t < rest)
            see((float)z[whole * E + t], v0 + whole * E + t);
        return b;
    };
    sh.best[tid] = best_of(tid, 0, 1, ~(uint64_t)0);
    for (int r = 0; r < k; ++r) {
        __syncthreads();
        if (tid < 64) {
            uint64_t b = 0;
            int who = 0;
            for (int i = tid; i < LP_THREADS; i += 64)
                if (sh.best[i] > b) {
                    b = sh.best[i];
                    who = i;
                }
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) {
                const uint64_t ob = __shfl_xor(b, o, 64);
                const int ow = __shfl_xor(who, o, 64);
                if (ob > b) {
                    b = ob;
                    who = ow;
                }
            }
            if (tid == 0) {
                sh.win = b;
                sh.n_threads = who;
                emit(r, b);
            }
        }
        __syncthreads();
        const uint64_t win = sh.win;
        const int who = sh.n_threads;
        // the winner's next, from all threads
        const uint64_t b = best_of(who, tid, LP_THREADS, win);
        if (tid == 0)
            sh.best[who] = 0;
        __syncthreads();
        if (b)
            atomicMax((unsigned long long *)&sh.best[who], (unsigned long long)b);
    }
}

// Sums of the threads' states over the workgroup, in every thread.
__device__ __forceinline__ LpState lp_sum(LpState t, float c, LpState *waves, int tid)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        LpState u;
        u.m = __shfl_xor(t.m, o, 64);
        u.s = __shfl_xor(t.s, o, 64);
        u.w = __shfl_xor(t.w, o, 64);
        t.join(u, c);
    }
    if ((tid & 63) == 0)
        waves[tid >> 6] = t;
    __syncthreads();
    LpState all{-INFINITY, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < LP_THREADS / 64; ++w)
        all.join(waves[w], c);
    return all;
}

// Whether one logit is above all others: its exponential is 1 itself.
__device__ __forceinline__ bool lp_confident(float s) { return s >= 1.f && s < 2.f; }

struct LpOthers {
    int who;
    float waves[LP_THREADS / 64];
};

// S - 1 of such a segment, in every thread: the threads' own sums relative to m, but
// for the thread `has`, whose logits (pieces tid, tid + 256, ... and one of the rest)
// all read again, without the largest.  Only such rows pay for it: 4096 x 131072 bf16
// of them take 170 us, others 166; 16000 x 1404, a wave each, 14.2 and 13.4.  (Counting
// the largest logits apart in every row's sums: 183 us and 17.4.)
template <typename TI, int E>
__device__ __forceinline__ float lp_others(const TI *z, int n, float m, float c, float own, bool has, LpOthers &sh, int tid)
{
    const int whole = n / E, rest = n - whole * E;
    if (has)
        sh.who = tid;
    __syncthreads();
    const int who = sh.who;
    float s = has ? 0.f : own;
    auto add = [&](float x) { s += x < m ? lp_exp2(lp_arg(x, m, c)) : 0.f; };
    for (int i = tid * LP_THREADS + who; i < whole; i += LP_THREADS * LP_THREADS) {
        RowPiece<TI, E> v;
        v.load(z + (int64_t)i * E);
#pragma unroll
        for (int e = 0; e < E; ++e)
            add(v.at(e));
    }
    if (tid == 0 && who < rest)
        add((float)z[whole * E + who]);
    s = wave_sum(s);
    if ((tid & 63) == 0)
        sh.waves[tid >> 6] = s;
    __syncthreads();
    s = sh.waves[0];
#pragma unroll
    for (int w = 1; w < LP_THREADS / 64; ++w)
        s += sh.waves[w];
    return s;
}

// ------------------------------------------------------------------ forward
// The token's logit of a row, and whether there is one: asked for before the row is
// read, used after.
template <typename TI> __device__ __forceinline__ bool lp_target(const LpArgs &p, int64_t t, float &z)
{
    if (!p.logp)
        return false;
    const int at = p.id64 ? token_key((const int64_t *)p.targets, t, p.V) : token_key((const int32_t *)p.targets, t, p.V);
    z = (float)((const TI *)p.logits)[t * p.ld + (at < p.V ? at : 0)];
    return at < p.V;
}

// One workgroup a row, or a segment of a row that is longer than LP_SEG.
// Bound by memory: 4096 x 131072 bf16 take 166 us (6.5 TB/s), with or without the
// entropy's operations.  ONCE: more than the caches behind the L2s hold, read past
// them (190 us through them; workgroups that start at different places of their
// rows 3% more, segments of 4096 a sixth more).
template <typename TI, bool TOP, bool ONCE> __global__ __launch_bounds__(LP_THREADS) void logprob_kernel(LpArgs p)
{
    constexpr int E = Elt<TI>::PER_CHUNK, U = 4;
    __shared__ LpState waves[LP_THREADS / 64];
    __shared__ LpOthers others;
    __shared__ __attribute__((aligned(16))) char top_mem[TOP ? sizeof(LpTop) : 16];
    const int tid = threadIdx.x;
    const int64_t t = blockIdx.x / p.segs;
    const int s = (int)(blockIdx.x - t * p.segs), v0 = s * p.seg;
    const int n = p.V - v0 < p.seg ? p.V - v0 : p.seg;
    const TI *z = (const TI *)p.logits + t * p.ld + v0;
    const float c = p.scale2;
    float target = 0.f;
    const bool given = tid == 0 && p.segs == 1 && lp_target<TI>(p, t, target);
    LpState st{-INFINITY, 0.f, 0.f};
    const int whole = n / E, rest = n - whole * E;
    for (int i = tid; i < whole; i += LP_THREADS * U) {
        RowPiece<TI, E> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i + u * LP_THREADS < whole)
                v[u].template load<ONCE>(z + (int64_t)(i + u * LP_THREADS) * E);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i + u * LP_THREADS < whole) {
                float top = v[u].at(0);
#pragma unroll
                for (int e = 1; e < E; ++e)
                    top = lp_max(top, v[u].at(e));
                if (!(top <= st.m))
                    st.raise(lp_max(top, st.m), c);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    st.add(v[u].at(e), c);
            }
    }
    if (tid < rest) {
        const float x = (float)z[whole * E + tid];
        if (!(x <= st.m))
            st.raise(lp_max(x, st.m), c);
        st.add(x, c);
    }
    const float largest = st.m, own = st.s;
    st = lp_sum(st, c, waves, tid);
    LpSum sum{st.m, st.s - 1.f, st.w};
    if (lp_confident(st.s))
        sum.more = lp_others<TI, E>(z, n, st.m, c, own * lp_exp2(lp_arg(largest, st.m, c)), largest == st.m, others, tid);
    if (tid == 0) {
        if (p.segs == 1)
            lp_finish(p, t, sum, given, target);
        else
            p.part[t * p.segs + s] = sum;
    }
    if constexpr (TOP) {
        LpTop &sh = *reinterpret_cast<LpTop *>(top_mem);
        auto own = [&](auto f) {
            for (int i = tid; i < whole; i += LP_THREADS) {
                RowPiece<TI, E> x;
                x.load(z + (int64_t)i * E);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    f(x.at(e), v0 + i * E + e);
            }
            if (tid < rest)
                f((float)z[whole * E + tid], v0 + whole * E + tid);
        };
        if (p.segs == 1) {
            const LpRow row(sum);
            lp_alternatives<TI, E>(z, v0, n, p.k, largest, own, sh, tid, [&](int r, uint64_t key) {
                p.top_idx[t * p.k + r] = row.bad ? r : lp_key_index(key);
                p.top_logp[t * p.k + r] = row.logp(lp_key_value(key), p.scale);
            });
        } else {
            uint64_t *keys = p.keys + (t * p.segs + s) * p.k;
            lp_alternatives<TI, E>(z, v0, n, p.k, largest, own, sh, tid, [&](int r, uint64_t key) { keys[r] = key; });
        }
    }
}

// One workgroup a row or a segment of at most LP_ONCE pieces a thread: rows too long for a wave,
// and few rows, where the time is that of one trip to memory and what follows.  The
// pieces are all requested at once; the segment's maximum comes before its
// exponentials, so that no sum is scaled.  32 segments of 4096 bf16 take 3 us, with
// 20 alternatives 7: the bound, the candidates' second read and their ranks.
template <typename TI, bool TOP> __global__ __launch_bounds__(LP_THREADS) void logprob_segment_kernel(LpArgs p)
{
    constexpr int E = Elt<TI>::PER_CHUNK, U = LP_ONCE, NW = LP_THREADS / 64;
    __shared__ float tops[NW];
    __shared__ LpState waves[NW];
    __shared__ LpOthers others;
    __shared__ __attribute__((aligned(16))) char top_mem[TOP ? sizeof(LpTop) : 16];
    const int tid = threadIdx.x, lane = tid & 63;
    const int64_t t = blockIdx.x / p.segs;
    const int s = (int)(blockIdx.x - t * p.segs), v0 = s * p.seg;
    const int n = p.V - v0 < p.seg ? p.V - v0 : p.seg;
    const TI *z = (const TI *)p.logits + t * p.ld + v0;
    const float c = p.scale2;
    float target = 0.f;
    const bool given = tid == 0 && p.segs == 1 && lp_target<TI>(p, t, target);
    const int whole = n / E, rest = n - whole * E;
    RowPiece<TI, E> v[U];
    float last = -INFINITY;
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (tid + u * LP_THREADS < whole)
            v[u].load(z + (tid + u * LP_THREADS) * E);
    if (tid < rest)
        last = (float)z[whole * E + tid];
    float largest = last;
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (tid + u * LP_THREADS < whole)
#pragma unroll
            for (int e = 0; e < E; ++e)
                largest = lp_max(largest, v[u].at(e));
    float top = largest;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        top = lp_max(top, __shfl_xor(top, o, 64));
    if (lane == 0)
        tops[tid >> 6] = top;
    __syncthreads();
    LpState st{lp_max(lp_max(tops[0], tops[1]), lp_max(tops[2], tops[3])), 0.f, 0.f};
    static_assert(NW == 4, "four waves");
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (tid + u * LP_THREADS < whole)
#pragma unroll
            for (int e = 0; e < E; ++e)
                st.add(v[u].at(e), c);
    if (tid < rest)
        st.add(last, c);
    const float own = st.s;
    st.s = wave_sum(st.s);
    st.w = wave_sum(st.w);
    if (lane == 0)
        waves[tid >> 6] = st;
    __syncthreads();
    st.s = waves[0].s + waves[1].s + waves[2].s + waves[3].s;
    LpSum sum{st.m, st.s - 1.f, waves[0].w + waves[1].w + waves[2].w + waves[3].w};
    if (lp_confident(st.s))
        sum.more = lp_others<TI, E>(z, n, st.m, c, own, largest == st.m, others, tid);
    if (tid == 0) {
        if (p.segs == 1)
            lp_finish(p, t, sum, given, target);
        else
            p.part[t * p.segs + s] = sum;
    }
    if constexpr (TOP) {
        LpTop &sh = *reinterpret_cast<LpTop *>(top_mem);
        auto own = [&](auto f) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (tid + u * LP_THREADS < whole)
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        f(v[u].at(e), v0 + (tid + u * LP_THREADS) * E + e);
            if (tid < rest)
                f(last, v0 + whole * E + tid);
        };
        if (p.segs == 1) {
            const LpRow row(sum);
            lp_alternatives<TI, E>(z, v0, n, p.k, largest, own, sh, tid, [&](int r, uint64_t key) {
                p.top_idx[t * p.k + r] = row.bad ? r : lp_key_index(key);
                p.top_logp[t * p.k + r] = row.logp(lp_key_value(key), p.scale);
            });
        } else {
            uint64_t *keys = p.keys + (t * p.segs + s) * p.k;
            lp_alternatives<TI, E>(z, v0, n, p.k, largest, own, sh, tid, [&](int r, uint64_t key) { keys[r] = key; });
        }
    }
}

// A wave's row of at most U pieces a lane, in registers: f(x, index, there) for every
// lane's elements, whether the row has them or not, a piece of every lane after another.
template <typename TI, int E, int U> struct LpLanes {
    RowPiece<TI, E> v[U];
    float last;
    int whole, rest, lane;
    __device__ __forceinline__ LpLanes(const TI *z, int n, int lane) : last(-INFINITY), whole(n / E), rest(n % E), lane(lane)
    {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (lane + u * 64 < whole)
                v[u].load(z + (lane + u * 64) * E);
        if (lane < rest)
            last = (float)z[whole * E + lane];
    }
    template <typename F> __device__ __forceinline__ void each(F f) const
    {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (u * 64 < whole) {
                const bool there = lane + u * 64 < whole;
#pragma unroll
                for (int e = 0; e < E; ++e)
                    f(there ? v[u].at(e) : -INFINITY, (lane + u * 64) * E + e, there);
            }
        if (rest)
            f(last, whole * E + lane, lane < rest);
    }
    // lp_others of the wave's row: the lane `has` has U E elements and one of the rest, read again by as many lanes.
    __device__ __forceinline__ float others(const TI *z, float m, float c, float own, bool has) const
    {
        static_assert(U * E <= 64, "an element a lane");
        const int i = __builtin_ctzll(__ballot(has)) + lane / E * 64;
        float s = has ? (last < m ? lp_exp2(lp_arg(last, m, c)) : 0.f) : own;
        if (lane < U * E && i < whole) {
            const float x = (float)z[i * E + lane % E];
            s += x < m ? lp_exp2(lp_arg(x, m, c)) : 0.f;
        }
        return wave_sum(s);
    }
    // How many elements pass a test, and the keys of the first `most` of them to a list.
    template <typename F> __device__ __forceinline__ int count(F test) const
    {
        int n = 0;
        each([&](float x, int, bool there) { n += __popcll(__ballot(there && test(x))); });
        return n;
    }
    template <typename F> __device__ __forceinline__ int list(uint64_t *to, int most, F test) const
    {
        int n = 0;
        each([&](float x, int v, bool there) {
            const bool hit = there && test(x);
            const uint64_t hits = __ballot(hit);
            if (hits) {
                const int at = n + __popcll(hits & ((1ull << lane) - 1));
                if (hit && at < most)
                    to[at] = lp_key(x, v);
                n += __popcll(hits);
            }
        });
        return n;
    }
};

// Orders the wave's writes to LDS and its reads of them.
__device__ __forceinline__ void lp_wave_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// The k best of a wave's row to emit(rank, key), best first; `largest`: of a lane's
// elements.  Of these, or where k is more than LP_WAVE_HEADS of the lanes' pieces, k have a
// largest that reaches the k-th largest: a bound that k logits reach (of 64 lanes the
// 64th lets 250 of 2048 pass, of their 256 pieces 80).  What reaches the bound is listed
// (masked logits only if there are too few others), and each compared with each.  Where
// that is much more than k (equal logits in bulk, all in few lanes), the k-th largest of
// all is found: it is the least that reaches the bound, unless k are above that; those
// are listed in their turn, and if they too are many the k-th is found bit by bit, from the
// list, or from the row where that is too short.  What is above it is listed, and as many
// equal to it as are wanted, the lowest indices first.
constexpr int LP_WAVE_CAND = 512, LP_WAVE_FEW = 96, LP_WAVE_HEADS = 24;
template <typename TI, int E, int U, typename F>
__device__ __forceinline__ void lp_wave_alternatives(const LpLanes<TI, E, U> &z, int k, float largest, uint64_t *list, F emit)
{
    constexpr int MINE = LP_WAVE_CAND / 64;
    const int lane = z.lane;
    const uint32_t lowest = lp_order(-INFINITY);
    // the largest order that k of many reach, or one below it, down to bit `last`: reach(order) counts them
    auto nth = [&](int last, auto reach) {
        uint32_t at = 0;
        for (int bit = 31; bit >= last; --bit) {
            const uint32_t up = at | 1u << bit;
            at = reach(up) >= k ? up : at;
        }
        return at < lowest ? lowest : at;
    };
    float bound = -INFINITY;
    if (k <= LP_WAVE_HEADS) {
        if (k <= (z.whole > z.rest ? z.whole : z.rest))
            bound = lp_value(lp_nth(lp_order(largest), k));
    } else if (k <= z.whole) {
        uint32_t head[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float top = z.v[u].at(0);
#pragma unroll
            for (int e = 1; e < E; ++e)
                top = lp_max(top, z.v[u].at(e));
            head[u] = lane + u * 64 < z.whole ? lp_order(top) : 0;
        }
        bound = lp_value(nth(12, [&](uint32_t least) {
            int n = 0;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (u * 64 < z.whole)
                    n += __popcll(__ballot(head[u] >= least));
            return n;
        }));
    }
    bound = fmaxf(bound, -__FLT_MAX__);  // (masked ones only if there are no others)
    int n = z.list(list, LP_WAVE_CAND, [&](float x) { return x >= bound; });
    lp_wave_fence();
    float least = -INFINITY;
    bool exact = n > LP_WAVE_FEW;
    if (exact) {
        least = INFINITY;
        z.each([&](float x, int, bool there) { least = there && x >= bound && x < least ? x : least; });
#pragma unroll
        for (int o = 32; o > 0; o >>= 1)
            least = fminf(least, __shfl_xor(least, o, 64));
        if (z.count([&](float x) { return x > least; }) >= k) {
            n = z.list(list, LP_WAVE_CAND, [&](float x) { return x > least; });
            lp_wave_fence();
            exact = n > LP_WAVE_FEW;
            if (n > LP_WAVE_CAND) {
                least = lp_value(nth(0, [&](uint32_t order) {
                    const float from = lp_value(order < lowest ? lowest : order);
                    return z.count([&](float x) { return x >= from; });
                }));
            } else if (exact) {
                uint32_t mine[MINE];
#pragma unroll
                for (int q = 0; q < MINE; ++q)
                    mine[q] = q * 64 + lane < n ? (uint32_t)(list[q * 64 + lane] >> 32) : 0;
                least = lp_value(nth(0, [&](uint32_t order) {
                    int reach = 0;
#pragma unroll
                    for (int q = 0; q < MINE; ++q)
                        if (q * 64 < n)
                            reach += __popcll(__ballot(mine[q] >= order));
                    return reach;
                }));
            }
        }
    }
    if (exact)
        n = z.list(list, LP_WAVE_CAND, [&](float x) { return x > least; });
    if (n < k) {
#pragma unroll
        for (int u = 0; u <= U; ++u) {
            if (n >= k)
                continue;
            uint32_t same = 0;
            if (u < U && lane + u * 64 < z.whole)
#pragma unroll
                for (int e = 0; e < E; ++e)
                    same |= (uint32_t)(z.v[u < U ? u : 0].at(e) == least) << e;
            if (u == U && lane < z.rest)
                same = z.last == least;
            if (!__ballot(same != 0))
                continue;
            int total;
            int to = n + wave_excl_scan(__popc(same), lane, total);
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (same >> e & 1 && to < k)
                    list[to++] = lp_key(least, (u < U ? (lane + u * 64) * E : z.whole * E + lane) + e);
            n = n + total < k ? n + total : k;
        }
    }
    lp_wave_fence();
    static_assert(LP_WAVE_FEW <= 128, "two keys a lane");
    const uint64_t a = lane < n ? list[lane] : 0, b = 64 + lane < n ? list[64 + lane] : 0;
    int above_a = a ? 0 : k, above_b = b ? 0 : k;
    if (n <= 64) {
#pragma unroll 16
        for (int j = 0; j < n; ++j)
            above_a += list[j] > a;
    } else {
#pragma unroll 16
        for (int j = 0; j < n; ++j) {
            const uint64_t other = list[j];
            above_a += other > a;
            above_b += other > b;
        }
    }
    if (above_a < k)
        emit(above_a, a);
    if (above_b < k)
        emit(above_b, b);
}

// One wave a row that it holds in registers: no barriers, and no sum is scaled.  16000 x
// 1404 bf16 take 13 us (3.4 TB/s), with 5 alternatives 20, with 64 42: a row's reductions,
// bounds and ranks take longer than its bytes.
template <typename TI, int U, bool TOP> __global__ __launch_bounds__(LP_THREADS) void logprob_wave_kernel(LpArgs p)
{
    constexpr int E = Elt<TI>::PER_CHUNK, NW = LP_THREADS / 64;
    __shared__ uint64_t lists[TOP ? NW : 1][TOP ? LP_WAVE_CAND : 1];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t = (int64_t)blockIdx.x * NW + wave;
    if (t >= p.T)
        return;
    const float c = p.scale2;
    float target = 0.f;
    const bool given = lane == 0 && lp_target<TI>(p, t, target);
    const LpLanes<TI, E, U> z((const TI *)p.logits + t * p.ld, p.V, lane);
    float largest = -INFINITY;
    z.each([&](float x, int, bool) { largest = lp_max(largest, x); });
    float top = largest;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        top = lp_max(top, __shfl_xor(top, o, 64));
    LpState st{top, 0.f, 0.f};
    z.each([&](float x, int, bool) { st.add(x, c); });
    const float all = wave_sum(st.s);
    LpSum sum{top, all - 1.f, wave_sum(st.w)};
    if (lp_confident(all))
        sum.more = z.others((const TI *)p.logits + t * p.ld, top, c, st.s, largest == top);
    if (lane == 0)
        lp_finish(p, t, sum, given, target);
    if constexpr (TOP) {
        const LpRow row(sum);
        auto emit = [&](int r, uint64_t key) {
            p.top_idx[t * p.k + r] = row.bad ? r : lp_key_index(key);
            p.top_logp[t * p.k + r] = row.logp(lp_key_value(key), p.scale);
        };
        if (row.bad) {
            if (lane < p.k)
                emit(lane, 0);
        } else {
            lp_wave_alternatives<TI, E, U>(z, p.k, largest, lists[wave], emit);
        }
    }
}

// The segments of a row joined: a lane a segment, in every wave.  The k best of
// their sorted lists: where r lists' entries number j reach a bound, r j keys do; the
// r-th largest of these entries, with r j >= k, is one, and the few keys that reach
// it are ranked.  2 us, with 20 alternatives 4.
template <typename TI, bool TOP> __global__ __launch_bounds__(LP_THREADS) void logprob_join_kernel(LpArgs p)
{
    constexpr int MOST = LP_MOST_TOP * LP_MOST_SEGS;
    __shared__ uint64_t cand[TOP ? MOST : 1];
    __shared__ int count;
    const int tid = threadIdx.x, lane = tid & 63;
    const int64_t t = blockIdx.x;
    const float c = p.scale2;
    const bool on = lane < p.segs;
    float target = 0.f;
    const bool given = tid == 0 && lp_target<TI>(p, t, target);
    LpSum sum = p.part[t * p.segs + (on ? lane : 0)];
    constexpr int EARLY = 4;  // keys a thread asks for before the bound is known
    const uint64_t *keys = nullptr;
    uint64_t early[EARLY];
    uint64_t entry_key = 0;
    int r = 0;
    if constexpr (TOP) {
        keys = p.keys + t * p.segs * p.k;
        int j = (2 * p.k + p.segs - 1) / p.segs;
        j = j < p.k ? j : p.k;
        r = (p.k + j - 1) / j;
        if (on)
            entry_key = keys[lane * p.k + j - 1];
#pragma unroll
        for (int q = 0; q < EARLY; ++q)
            early[q] = tid + q * LP_THREADS < p.segs * p.k ? keys[tid + q * LP_THREADS] : 0;
        if (tid == 0)
            count = 0;
    }
    LpState st{on ? sum.m : -INFINITY, on ? 1.f + sum.more : 0.f, on ? sum.w : 0.f};
    float top = st.m;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        top = lp_max(top, __shfl_xor(top, o, 64));
    const bool largest = st.m == top;
    const float more = sum.more;
    st.raise(top, c);
    const float all = wave_sum(st.s);
    sum = LpSum{top, all - 1.f, wave_sum(st.w)};
    if (lp_confident(all))  // the segment that has the largest logit, without it, and the others
        sum.more = wave_sum(largest ? more : st.s);
    if (tid == 0)
        lp_finish(p, t, sum, given, target);
    if constexpr (TOP) {
        const LpRow row(sum);
        if (row.bad) {
            for (int i = tid; i < p.k; i += LP_THREADS) {
                p.top_idx[t * p.k + i] = i;
                p.top_logp[t * p.k + i] = row.logp(0.f, 1.f);
            }
            return;
        }
        const uint32_t entry = (uint32_t)(entry_key >> 32);
        // (an order of 0 is no key's: one below all of them where a list is shorter than j)
        const uint64_t bound = (uint64_t)lp_nth(entry, r) << 32 | 1;
        __syncthreads();
        auto list = [&](uint64_t least) {
            auto offer = [&](uint64_t key) {
                if (key >= least)
                    cand[atomicAdd(&count, 1)] = key;
            };
#pragma unroll
            for (int q = 0; q < EARLY; ++q)
                offer(early[q]);
            for (int i = tid + EARLY * LP_THREADS; i < p.segs * p.k; i += LP_THREADS)
                offer(keys[i]);
            __syncthreads();
        };
        list(bound);
        if (count > LP_MANY) {  // equal logits in bulk: of the lists' entries with that order, the one with the r-th key
            const uint32_t order = (uint32_t)(bound >> 32);
            const int above = __popcll(__ballot(on && entry > order));
            const uint32_t low = on && entry == order ? (uint32_t)entry_key : 0;
            uint64_t exact = (uint64_t)order << 32 | lp_nth(low, r - above);
            // and a list's last entry is a bound that it reaches by itself
            const uint64_t end = on ? keys[lane * p.k + p.k - 1] : 0;
            const uint32_t high = lp_nth((uint32_t)(end >> 32), 1);
            const uint64_t last = (uint64_t)high << 32 | lp_nth((uint32_t)(end >> 32) == high ? (uint32_t)end : 0, 1);
            exact = last > exact ? last : exact;
            __syncthreads();
            if (tid == 0)
                count = 0;
            __syncthreads();
            list(exact > 0 ? exact : 1);
        }
        lp_rank(cand, count, p.k, tid, [&](int rank, uint64_t key) {
            p.top_idx[t * p.k + rank] = lp_key_index(key);
            p.top_logp[t * p.k + rank] = row.logp(lp_key_value(key), p.scale);
        });
    }
}

// ------------------------------------------------------------------ backward
// One workgroup a chunk of a row.  Every thread has read all of its elements
// before it writes them: dlogits may be logits.  Bound by memory: 4096 x 131072 bf16
// with the entropy's gradient 360 us (5.9 TB/s).
constexpr int LP_BACK_U = 4;
template <typename TI> __global__ __launch_bounds__(LP_THREADS) void logprob_backward_kernel(LpArgs p)
{
    constexpr int E = Elt<TI>::PER_CHUNK, U = LP_BACK_U;
    const int tid = threadIdx.x;
    const int64_t t = blockIdx.x / p.segs;
    const int v0 = (int)(blockIdx.x - t * p.segs) * p.seg;
    const int n = p.V - v0 < p.seg ? p.V - v0 : p.seg;
    const TI *z = (const TI *)p.logits + t * p.ld + v0;
    TI *o = (TI *)p.dlogits + t * p.ldd + v0;
    const float m = p.norm_in[2 * t], size = p.norm_in[2 * t + 1];
    const bool empty = m == -INFINITY;
    int at = p.V;
    if (p.dlogp)
        at = p.id64 ? token_key((const int64_t *)p.targets, t, p.V) : token_key((const int32_t *)p.targets, t, p.V);
    // dz = p (a + b log2 p), at the target p (a0 + b log2 p) + d (1 - p)
    const float h = p.dentropy ? p.dentropy[t] * p.scale : 0.f;
    const float d = at < p.V && !empty ? p.dlogp[t] * p.scale : 0.f;
    float a0 = p.dentropy && !empty ? -h * p.entropy_in[t] : 0.f;
    const float b = empty ? 0.f : -h * LP_LN2;
    if (size != size)
        a0 = size;
    const float a = a0 - d;
    const float base = empty ? 0.f : m, size2 = size * LP_LOG2E;
    auto grad = [&](float x) {
        const float l = fmaxf(fmaf(x - base, p.scale2, -size2), LP_LEAST);
        return lp_exp2(l) * fmaf(b, l, a);
    };
    auto grad_target = [&](float x) {  // (1 - p of a likely token would lose its digits)
        const float l = fmaxf(fmaf(x - base, p.scale2, -size2), LP_LEAST);
        return fmaf(-d, expm1f(l * LP_LN2), lp_exp2(l) * fmaf(b, l, a0));
    };
    const int whole = n / E, rest = n - whole * E;
    at -= v0;
    RowPiece<TI, E> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (tid + u * LP_THREADS < whole)
            v[u].load(z + (tid + u * LP_THREADS) * E);
    TI last{};
    if (tid < rest)
        last = z[whole * E + tid];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int i = (tid + u * LP_THREADS) * E;
        if (i / E < whole) {
            float g[E];
#pragma unroll
            for (int e = 0; e < E; ++e)
                g[e] = grad(v[u].at(e));
            if (at >= i && at < i + E) {
                float x = 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e)
                    x = at == i + e ? v[u].at(e) : x;
                x = grad_target(x);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    g[e] = at == i + e ? x : g[e];
            }
            rows_store<E>(o + i, g, 0);
        }
    }
    if (tid < rest)
        o[whole * E + tid] = (TI)(at == whole * E + tid ? grad_target((float)last) : grad((float)last));
}

// ------------------------------------------------------------------ host
static int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Few rows are cut into segments, so that LP_WGS workgroups have work: of LP_SEG
// logits at most, where LP_MOST_SEGS of them are enough.  A row of up to LP_WHOLE
// bytes takes one workgroup less time than the second launch that joins segments (4
// us).
constexpr int LP_WGS = 1024, LP_WHOLE = 48 << 10;

// Rows that one wave takes: of up to LP_WAVE_SMALL pieces a lane at any number (64 x 536
// fp32 with 5 alternatives 4.9 us, a workgroup a row 5.6; 16000 x 1404 bf16 20 and 51,
// with 64 alternatives 42 and 85; slower for few rows with 64, 64 x 1404 10.0 and 8.8: a
// row's sums are not to depend on how many are asked for), of up to LP_WAVE_MORE from
// LP_WAVE_ROWS on (5: 1024 x 4096 bf16 8.2 and 8.0 us, 2048 11.7 and 13.3, 16000 39 and 62).
// Twice as many pieces are slower at any number (16000 x 8000 bf16 109 and 73 us).
constexpr int LP_WAVE_ROWS = 2048, LP_WAVE_SMALL = 4, LP_WAVE_MORE = 8;

static int most_segments(int V)
{
    const int64_t n = ceil_div(V, LP_SEG);
    return (int)(n < LP_MOST_SEGS ? n : LP_MOST_SEGS);
}

void lp_segments(int T, int V, int bf16, int &segs, int &seg)
{
    const bool whole = (int64_t)V * (bf16 ? 2 : 4) <= LP_WHOLE;
    const int64_t want = T > 0 && !whole ? ceil_div(LP_WGS, T) : 1, most = most_segments(V);
    const int64_t n = want < most ? want : most;
    seg = (int)(ceil_div(ceil_div(V, n), 8) * 8);
    segs = (int)ceil_div(V, seg);
}

static size_t bytes_of(int64_t parts, int k) { return (size_t)parts * (sizeof(LpSum) + (size_t)k * 8); }

size_t lp_workspace(int T, int V, int bf16, int k)
{
    int segs, seg;
    lp_segments(T, V, bf16, segs, seg);
    return segs > 1 ? bytes_of((int64_t)T * segs, k) : 0;
}

// Rows t times segments, of either type: at most most_segments(V) each, and below LP_WGS + t.
size_t lp_most_workspace(int T, int V, int k)
{
    const int64_t t = T < LP_WGS ? T : LP_WGS - 1, most = most_segments(V);
    if ((int64_t)V * 4 <= LP_WHOLE)
        return 0;
    const int64_t a = t * most, b = LP_WGS + t;
    return bytes_of(a < b ? a : b, k);
}

// A launch's threads are counted in 32 bits: workgroups that it has at most.  More rows take further launches.
constexpr int64_t LP_GRID = ((int64_t)1 << 32) / LP_THREADS - 1;

// The call's rows from t0 on, at most `most`.
static LpArgs lp_rows(const LpArgs &a, int64_t t0, int64_t most)
{
    const int es = a.bf16 ? 2 : 4;
    LpArgs p = a;
    auto on = [&](auto &q, int64_t step) {
        if (q)
            q += t0 * step;
    };
    auto bytes_on = [&](auto &q, int64_t step) {
        if (q)
            q = (std::remove_reference_t<decltype(q)>)((uintptr_t)q + t0 * step);
    };
    p.T = (int)(a.T - t0 < most ? a.T - t0 : most);
    bytes_on(p.logits, a.ld * es);
    bytes_on(p.dlogits, a.ldd * es);
    bytes_on(p.targets, a.id64 ? 8 : 4);
    on(p.logp, 1);
    on(p.norm, 2);
    on(p.entropy, 1);
    on(p.top_logp, a.k);
    on(p.top_idx, a.k);
    on(p.norm_in, 2);
    on(p.entropy_in, 1);
    on(p.dlogp, 1);
    on(p.dentropy, 1);
    return p;
}

static hipError_t run_logprob(LpArgs p, void *ws, hipStream_t s)
{
    if (p.segs > 1) {
        p.keys = (uint64_t *)ws;
        p.part = (LpSum *)(p.keys + (int64_t)p.T * p.segs * p.k);
    }
    const dim3 grid((unsigned)((int64_t)p.T * p.segs)), block(LP_THREADS);
    auto run = [&](auto type, auto top) {
        using TI = decltype(type);
        constexpr bool TOP = decltype(top)::value;
        const dim3 waves((unsigned)ceil_div(p.T, LP_THREADS / 64));
        const int pieces = p.V / Elt<TI>::PER_CHUNK;
        if (pieces <= 64 * LP_WAVE_SMALL)
            logprob_wave_kernel<TI, LP_WAVE_SMALL, TOP><<<waves, block, 0, s>>>(p);
        else if (pieces <= 64 * LP_WAVE_MORE && p.T >= LP_WAVE_ROWS)
            logprob_wave_kernel<TI, LP_WAVE_MORE, TOP><<<waves, block, 0, s>>>(p);
        else if (p.seg <= LP_THREADS * LP_ONCE * Elt<TI>::PER_CHUNK)
            logprob_segment_kernel<TI, TOP><<<grid, block, 0, s>>>(p);
        else if (!TOP && (int64_t)p.T * p.V * (int64_t)sizeof(TI) > ((int64_t)256 << 20))
            logprob_kernel<TI, TOP, true><<<grid, block, 0, s>>>(p);
        else
            logprob_kernel<TI, TOP, false><<<grid, block, 0, s>>>(p);
    };
    if (p.bf16)
        p.k ? run(__bf16{}, std::true_type{}) : run(__bf16{}, std::false_type{});
    else
        p.k ? run(float{}, std::true_type{}) : run(float{}, std::false_type{});
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.segs == 1)
        return e;
    const dim3 rows((unsigned)p.T);
    if (p.bf16)
        p.k ? logprob_join_kernel<__bf16, true><<<rows, block, 0, s>>>(p)
            : logprob_join_kernel<__bf16, false><<<rows, block, 0, s>>>(p);
    else
        p.k ? logprob_join_kernel<float, true><<<rows, block, 0, s>>>(p)
            : logprob_join_kernel<float, false><<<rows, block, 0, s>>>(p);
    return hipGetLastError();
}

hipError_t launch_logprob(const LpArgs &args, void *ws, hipStream_t s)
{
    LpArgs p = args;
    p.scale2 = p.scale * LP_LOG2E;
    lp_segments(p.T, p.V, p.bf16, p.segs, p.seg);
    for (int64_t t0 = 0; t0 < p.T; t0 += LP_GRID) {  // (rows in segments are fewer than LP_WGS)
        const hipError_t e = run_logprob(lp_rows(p, t0, LP_GRID), ws, s);
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

hipError_t launch_logprob_backward(const LpArgs &args, hipStream_t s)
{
    LpArgs all = args;
    all.scale2 = all.scale * LP_LOG2E;
    all.seg = LP_THREADS * LP_BACK_U * (all.bf16 ? 8 : 4);
    all.segs = (int)ceil_div(all.V, all.seg);
    const int64_t most = LP_GRID / all.segs;
    for (int64_t t0 = 0; t0 < all.T; t0 += most) {
        const LpArgs p = lp_rows(all, t0, most);
        const dim3 grid((unsigned)((int64_t)p.T * p.segs)), block(LP_THREADS);
        if (p.bf16)
            logprob_backward_kernel<__bf16><<<grid, block, 0, s>>>(p);
        else
            logprob_backward_kernel<float><<<grid, block, 0, s>>>(p);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

}  // namespace twell
