// capi_tokens.cpp -- the C ABI of the operators at a model's two ends
// (include/twell.h): argument checks on the host, then launches on the caller's
// stream.
#include "twell.h"

#include <cmath>

#include <hip/hip_runtime.h>

#include "checks.h"
#include "embed.h"
#include "logprob.h"

namespace {

constexpr int32_t MOST_TOKENS = 1 << 30;  // of a vocabulary: keys up to V, and one more, stay below 2^31

int check_ids(const void *ids, int32_t id_bits) { return check_vec(ids, id_bits / 8); }

// Sizes of the embedding calls: the lookup's threads, of 4 pieces of 4 columns each (below 4: of one), are counted in 32
// bits.
int check_embed(int32_t T, int32_t V, int32_t d)
{
    if (T < 0 || T > MOST_ROWS || V < 1 || V > MOST_TOKENS || d < 1 || d > (1 << 20))
        return TWELL_E_SHAPE;
    return (int64_t)T * (d < 4 ? d : (d + 3) / 4) <= (((int64_t)1 << 24) - 1) * 1024 ? TWELL_OK : TWELL_E_SHAPE;
}

// Sizes of the log probabilities: rows times pieces of 2048 logits stay below 2^31.
int check_logprob(int32_t T, int32_t V, int32_t k)
{
    if (T < 0 || T > MOST_ROWS || V < 1 || V > MOST_TOKENS || k < 0 || k > V)
        return TWELL_E_SHAPE;
    if (k > twell::LP_MOST_TOP)
        return TWELL_E_UNSUPPORTED;
    return (int64_t)T * (((int64_t)V + 2047) / 2048) < ((int64_t)1 << 31) ? TWELL_OK : TWELL_E_SHAPE;
}

// Whether rows of `row` bytes at `b` lie apart from those at `a`, or in their place: rows ld and ldd bytes apart.
bool apart(const void *a, int64_t ld, const void *b, int64_t ldd, int64_t T, int64_t row)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    if (x == y)
        return ld == ldd || T == 1;
    if (x + (T - 1) * ld + row <= y || y + (T - 1) * ldd + row <= x)
        return true;
    if (ld != ldd)
        return false;
    const uintptr_t off = (y > x ? y - x : x - y) % (uintptr_t)ld;  // side by side in one buffer
    return off >= (uintptr_t)row && off + (uintptr_t)row <= (uintptr_t)ld;
}

// The kernels take the scale times log2(e): infinite, it would make the largest logit's exponential that of no number.
bool good_scale(float scale) { return scale > 0 && std::isfinite(scale * 1.44269504f); }
bool known_ids(int32_t id_bits) { return id_bits == 32 || id_bits == 64; }

}  // namespace

extern "C" {

int twell_embed_forward(const void *ids, int32_t id_bits, int32_t T, const void *table, int32_t V, int32_t d,
                        int32_t vdtype, float scale, void *out, int32_t odtype, void *stream)
{
    if (!known_dtype(vdtype) || !known_dtype(odtype) || !known_ids(id_bits))
        return TWELL_E_UNSUPPORTED;
    TWELL_TRY(check_embed(T, V, d));
    if (T == 0)
        return TWELL_OK;
    TWELL_TRY(check_ids(ids, id_bits));
    TWELL_TRY(check_vec(table, elem_size(vdtype)));
    TWELL_TRY(check_vec(out, elem_size(odtype)));
    const int64_t written = (int64_t)T * d * elem_size(odtype);
    if (overlap(out, written, table, (int64_t)V * d * elem_size(vdtype)) || overlap(out, written, ids, (int64_t)T * (id_bits / 8)))
        return TWELL_E_SHAPE;
    twell::EmbArgs a{};
    a.T = T;
    a.V = V;
    a.d = d;
    a.id64 = id_bits == 64;
    a.bf16_rows = odtype == TWELL_BF16;
    a.bf16_table = vdtype == TWELL_BF16;
    a.scale = scale;
    a.ids = ids;
    a.in = table;
    a.out = out;
    return hip_status(twell::launch_embed(a, static_cast<hipStream_t>(stream)));
}

size_t twell_embed_workspace_bytes(int32_t T, int32_t V, int32_t d)
{
    if (check_embed(T, V, d) != TWELL_OK)
        return 0;
    twell::EmbArgs a{};
    a.T = T;
    a.V = V;
    a.d = d;
    return twell::emb_layout(a, nullptr);
}

int twell_embed_backward(const void *ids, int32_t id_bits, int32_t T, const void *dout, int32_t dodtype, int32_t V,
                         int32_t d, float scale, int32_t accumulate, void *dtable, int32_t vdtype, void *workspace,
                         size_t workspace_bytes, void *stream)
{
    if (!known_dtype(vdtype) || !known_dtype(dodtype) || !known_ids(id_bits))
        return TWELL_E_UNSUPPORTED;
    TWELL_TRY(check_embed(T, V, d));
    if (T > 0) {
        TWELL_TRY(check_ids(ids, id_bits));
        TWELL_TRY(check_vec(dout, elem_size(dodtype)));
    }
    TWELL_TRY(check_vec(dtable, elem_size(vdtype)));
    twell::EmbArgs a{};
    a.T = T;
    a.V = V;
    a.d = d;
    a.id64 = id_bits == 64;
    a.bf16_rows = dodtype == TWELL_BF16;
    a.bf16_table = vdtype == TWELL_BF16;
    a.accumulate = accumulate != 0;
    a.scale = scale;
    a.ids = ids;
    a.in = dout;
    a.out = dtable;
    TWELL_TRY(check_ws(workspace, workspace_bytes, twell::emb_layout(a, workspace)));
    const int64_t written = (int64_t)V * d * elem_size(vdtype);
    if (overlap(dtable, written, dout, (int64_t)T * d * elem_size(dodtype)) ||
        overlap(dtable, written, ids, (int64_t)T * (id_bits / 8)))
        return TWELL_E_SHAPE;
    return hip_status(twell::launch_embed_backward(a, static_cast<hipStream_t>(stream)));
}

size_t twell_logprob_workspace_bytes(int32_t T, int32_t V, int32_t k)
{
    return check_logprob(T, V, k) == TWELL_OK ? twell::lp_most_workspace(T, V, k) : 0;
}

int twell_logprob_forward(const void *logits, int64_t ld, int32_t T, int32_t V, int32_t vdtype, float scale,
                          const void *targets, int32_t id_bits, float *logp, float *norm, float *entropy,
                          float *top_logp, int32_t *top_idx, int32_t k, void *workspace, size_t workspace_bytes,
                          void *stream)
{
    if (!known_dtype(vdtype) || !known_ids(id_bits))
        return TWELL_E_UNSUPPORTED;
    TWELL_TRY(check_logprob(T, V, k));
    if (ld < V || ld > ((int64_t)1 << 40) || !good_scale(scale))
        return TWELL_E_SHAPE;
    if (T == 0)
        return TWELL_OK;
    TWELL_TRY(check_vec(logits, elem_size(vdtype)));
    if (!logp && !norm && !entropy && !k)
        return TWELL_E_NULL;
    if (logp)
        TWELL_TRY(check_ids(targets, id_bits));
    for (const void *p : {(const void *)logp, (const void *)norm, (const void *)entropy})
        if (!aligned_to(p, 4))
            return TWELL_E_ALIGN;
    if (k) {
        TWELL_TRY(check_vec(top_logp, 4));
        TWELL_TRY(check_vec(top_idx, 4));
    }
    TWELL_TRY(check_ws(workspace, workspace_bytes, twell::lp_workspace(T, V, vdtype == TWELL_BF16, k)));
    twell::LpArgs a{};
    a.T = T;
    a.V = V;
    a.k = k;
    a.id64 = id_bits == 64;
    a.bf16 = vdtype == TWELL_BF16;
    a.scale = scale;
    a.ld = ld;
    a.logits = logits;
    a.targets = targets;
    a.logp = logp;
    a.norm = norm;
    a.entropy = entropy;
    a.top_logp = top_logp;
    a.top_idx = top_idx;
    return hip_status(twell::launch_logprob(a, workspace, static_cast<hipStream_t>(stream)));
}

int twell_logprob_backward(const void *logits, int64_t ld, int32_t T, int32_t V, int32_t vdtype, float scale,
                           const void *targets, int32_t id_bits, const float *norm, const float *entropy,
                           const float *dlogp, const float *dentropy, void *dlogits, int64_t ldd, void *stream)
{
    if (!known_dtype(vdtype) || !known_ids(id_bits))
        return TWELL_E_UNSUPPORTED;
    TWELL_TRY(check_logprob(T, V, 0));
    if (ld < V || ldd < V || ld > ((int64_t)1 << 40) || ldd > ((int64_t)1 << 40) || !good_scale(scale))
        return TWELL_E_SHAPE;
    if (T == 0)
        return TWELL_OK;
    TWELL_TRY(check_vec(logits, elem_size(vdtype)));
    TWELL_TRY(check_vec(dlogits, elem_size(vdtype)));
    const int es = elem_size(vdtype);
    if (!apart(logits, ld * es, dlogits, ldd * es, T, (int64_t)V * es))
        return TWELL_E_SHAPE;
    TWELL_TRY(check_vec(norm, 4));
    if (!dlogp && !dentropy)
        return TWELL_E_NULL;
    if (dlogp) {
        TWELL_TRY(check_vec(dlogp, 4));
        TWELL_TRY(check_ids(targets, id_bits));
    }
    if (dentropy) {
        TWELL_TRY(check_vec(dentropy, 4));
        TWELL_TRY(check_vec(entropy, 4));
    }
    twell::LpArgs a{};
    a.T = T;
    a.V = V;
    a.id64 = id_bits == 64;
    a.bf16 = vdtype == TWELL_BF16;
    a.scale = scale;
    a.ld = ld;
    a.ldd = ldd;
    a.logits = logits;
    a.targets = targets;
    a.norm_in = norm;
    a.entropy_in = entropy;
    a.dlogp = dlogp;
    a.dentropy = dentropy;
    a.dlogits = dlogits;
    return hip_status(twell::launch_logprob_backward(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
