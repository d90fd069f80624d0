// capi_dense.cpp -- the C ABI of the dense layer's operators (include/twell.h):
// argument checks on the host, then launches on the caller's stream.
#include "twell.h"

#include <cmath>

#include <hip/hip_runtime.h>

#include "act8.h"
#include "adamw.h"
#include "block_norm.h"
#include "checks.h"
#include "glu.h"

namespace {

// Sizes and types of the gated product.
int check_glu(int32_t T, int32_t d, int32_t F, int32_t vdtype, int32_t act)
{
    if (!known_dtype(vdtype) || act < TWELL_ACT_RELU || act > TWELL_ACT_GELU_TANH)
        return TWELL_E_UNSUPPORTED;
    if (T < 0 || T > MOST_ROWS || d <= 0 || F <= 0 || d % 64 != 0 || F % 64 != 0)
        return TWELL_E_SHAPE;
    // a tile's rows are addressed with 32-bit offsets
    if (d > (1 << 20) || F > (1 << 19))
        return TWELL_E_UNSUPPORTED;
    // workgroups of 64 x 64 results, split up to 16 times
    return ((int64_t)T + 63) / 64 * (F / 64 > d / 64 ? F / 64 : d / 64) * 16 < ((int64_t)1 << 31) ? TWELL_OK : TWELL_E_SHAPE;
}

// Codes and scales of 8-bit activations.
int check_packed(const twell_packed_t *p, size_t code_align)
{
    if (!p)
        return TWELL_E_NULL;
    TWELL_TRY(check_vec(p->code, code_align));
    return check_vec(p->scale, 2);
}

twell::Packed8 packed8(const twell_packed_t *p) { return twell::Packed8{p->code, static_cast<uint16_t *>(p->scale)}; }

// Whether T rows of d codes, or their scales, lie in part in `rows` of elements of that type.
bool packed_overlaps(const twell_packed_t *p, const void *rows, int32_t T, int32_t d, int32_t vdtype)
{
    const int64_t bytes = (int64_t)T * d * elem_size(vdtype), scales = T * twell::a8_blocks(d) * 2;
    return overlap(p->code, (int64_t)T * d, rows, bytes) || overlap(p->scale, scales, rows, bytes);
}

// Sizes of rows that are packed: the threads, of 2 pieces of 16 bytes each, are counted in 32 bits.
int check_act(int32_t T, int32_t d, int32_t vdtype)
{
    if (!known_dtype(vdtype))
        return TWELL_E_UNSUPPORTED;
    if (T < 0 || T > MOST_ROWS || d < 1 || d > (1 << 20))
        return TWELL_E_SHAPE;
    const int64_t pieces = T * twell::a8_blocks(d) * (vdtype == TWELL_BF16 ? 4 : 8);
    return pieces <= (((int64_t)1 << 24) - 1) * 512 ? TWELL_OK : TWELL_E_SHAPE;
}

// The descriptor of the block norms, and with `gated` its gate pointer.
int check_block_norm(const twell_block_norm_t *bn, bool gated)
{
    if (!bn)
        return TWELL_E_NULL;
    if ((bn->kind != TWELL_NORM_RMS && bn->kind != TWELL_NORM_LAYER) || !known_dtype(bn->rdtype) ||
        !known_dtype(bn->ydtype) || !known_dtype(bn->ndtype) || !known_dtype(bn->wdtype) ||
        bn->d > twell::BN_MAX_D)
        return TWELL_E_UNSUPPORTED;
    if (bn->T < 0 || bn->T > MOST_ROWS || bn->d < 1 || bn->gate_span < 0 || !(bn->eps > 0))
        return TWELL_E_SHAPE;
    for (const void *w : {bn->w_post, bn->b_post, bn->w_pre, bn->b_pre})
        if (w)
            TWELL_TRY(check_vec(w, elem_size(bn->wdtype)));
    return gated && bn->T > 0 ? check_vec(bn->gate, elem_size(bn->rdtype)) : TWELL_OK;
}

twell::BnTensor bn_tensor(const void *p, int32_t dt) { return twell::BnTensor{const_cast<void *>(p), dt == TWELL_BF16}; }

twell::BnArgs bn_args(const twell_block_norm_t *bn, bool block)
{
    twell::BnArgs a{};
    a.T = bn->T;
    a.d = bn->d;
    a.post = block && bn->post;
    a.eps = bn->eps;
    a.alpha = bn->alpha;
    a.gate_span = block ? bn->gate_span : 0;
    a.gate = bn_tensor(a.gate_span ? bn->gate : nullptr, bn->rdtype);
    a.w_post = bn_tensor(a.post ? bn->w_post : nullptr, bn->wdtype);
    a.b_post = bn_tensor(a.post ? bn->b_post : nullptr, bn->wdtype);
    a.w_pre = bn_tensor(bn->w_pre, bn->wdtype);
    a.b_pre = bn_tensor(bn->b_pre, bn->wdtype);
    return a;
}

// Whether every row of every tensor starts at a 16-byte boundary.
bool bn_wide(const twell::BnArgs &a)
{
    bool ok = a.d % 8 == 0;
    for (const twell::BnTensor *t : {&a.res, &a.y, &a.gate, &a.out, &a.n, &a.w_post, &a.b_post, &a.w_pre, &a.b_pre,
                                     &a.dout, &a.dn, &a.dres, &a.dy, &a.dgate})
        ok = ok && aligned16(t->p);
    return ok;
}

// One descriptor of twell_adamw_step (grads) or twell_adamw_unpack (values).
int check_adamw(const twell_adamw_tensor_t &t, bool coded, bool unpack)
{
    if (t.n < 0 || t.n > ((int64_t)1 << 40))
        return TWELL_E_SHAPE;
    if (!unpack && (!known_dtype(t.pdtype) || !known_dtype(t.gdtype)))
        return TWELL_E_UNSUPPORTED;
    if (t.n == 0)
        return TWELL_OK;
    TWELL_TRY(check_vec(t.m, coded ? 1 : 4));
    TWELL_TRY(check_vec(t.v, coded ? 1 : 4));
    if (coded) {
        TWELL_TRY(check_vec(t.m_scale, 4));
        TWELL_TRY(check_vec(t.v_scale, 4));
    }
    if (unpack) {
        TWELL_TRY(check_vec(t.m_values, 4));
        return check_vec(t.v_values, 4);
    }
    TWELL_TRY(check_vec(t.p, elem_size(t.pdtype)));
    TWELL_TRY(check_vec(t.grad, elem_size(t.gdtype)));
    return t.copy ? check_vec(t.copy, 2) : TWELL_OK;
}

// A launch's workgroups fit a grid.
constexpr int64_t AW_MOST_CHUNKS = (int64_t)1 << 30;
int64_t aw_chunks(int64_t n, int passes) { return (n + passes * twell::AW_PASS - 1) / (passes * twell::AW_PASS); }

// Passes of a workgroup: AW_PASSES (fewer searches for the tensor), but one
// where the call's elements would then leave some of the 256 CUs idle.
int aw_passes(const twell_adamw_tensor_t *tensors, int32_t count)
{
    int64_t chunks = 0;
    for (int32_t i = 0; i < count; ++i)
        chunks += aw_chunks(tensors[i].n, twell::AW_PASSES);
    return chunks < 256 ? 1 : twell::AW_PASSES;
}

}  // namespace

extern "C" {

size_t twell_glu_workspace_bytes(int32_t T, int32_t d, int32_t F, int32_t vdtype)
{
    return check_glu(T, d, F, vdtype, TWELL_ACT_RELU) == TWELL_OK ? twell::glu_forward_most_ws(T, d, F, vdtype, false) : 0;
}

int twell_glu_forward(const void *x, const void *wg_t, const void *wu_t, int32_t T, int32_t d, int32_t F,
                      int32_t vdtype, int32_t act, void *h, void *g, void *u, void *workspace, size_t workspace_bytes,
                      void *stream)
{
    TWELL_TRY(check_glu(T, d, F, vdtype, act));
    if (T == 0)
        return TWELL_OK;
    TWELL_TRY(check_mat(x));
    TWELL_TRY(check_mat(wg_t));
    TWELL_TRY(check_mat(wu_t));
    TWELL_TRY(check_mat(h));
    if (!aligned16(g) || !aligned16(u))
        return TWELL_E_ALIGN;
    TWELL_TRY(check_ws(workspace, workspace_bytes, twell::glu_forward_ws(T, d, F, vdtype, false)));
    twell::GluFwd a{};
    a.T = T;
    a.d = d;
    a.F = F;
    a.act = act;
    a.x = x;
    a.wg = wg_t;
    a.wu = wu_t;
    a.h = h;
    a.g = g;
    a.u = u;
    a.part = static_cast<float *>(workspace);
    return hip_status(twell::launch_glu(vdtype, a, static_cast<hipStream_t>(stream)));
}

size_t twell_glu_backward_workspace_bytes(int32_t T, int32_t d, int32_t F, int32_t vdtype)
{
    return check_glu(T, d, F, vdtype, TWELL_ACT_RELU) == TWELL_OK ? twell::glu_backward_most_ws(T, d, F, vdtype) : 0;
}

int twell_glu_backward(const void *x, const void *wg_t, const void *wu_t, const void *g, const void *u, const void *dh,
                       int32_t T, int32_t d, int32_t F, int32_t vdtype, int32_t act, void *dx, void *dwg, void *dwu,
                       void *workspace, size_t workspace_bytes, void *stream)
{
    TWELL_TRY(check_glu(T, d, F, vdtype, act));
    if (T > 0) {
        for (const void *p : {x, wg_t, wu_t, g, u, dh})
            TWELL_TRY(check_mat(p));
        if (!dx && !dwg)
            return TWELL_E_NULL;
    }
    if (!dwg != !dwu)
        return TWELL_E_NULL;
    if (!aligned16(dx) || !aligned16(dwg) || !aligned16(dwu))
        return TWELL_E_ALIGN;
    const twell::GluWs w = twell::glu_backward_ws(T, d, F, vdtype);
    TWELL_TRY(check_ws(workspace, workspace_bytes, w.bytes));
    twell::GluBwd a{};
    a.T = T;
    a.d = d;
    a.F = F;
    a.act = act;
    a.x = x;
    a.wg = wg_t;
    a.wu = wu_t;
    a.g = g;
    a.u = u;
    a.dh = dh;
    a.dx = dx;
    a.dwg = dwg;
    a.dwu = dwu;
    a.dgu = workspace;
    a.ws = w;
    return hip_status(twell::launch_glu_backward(vdtype, a, static_cast<hipStream_t>(stream)));
}

size_t twell_glu_packed_workspace_bytes(int32_t T, int32_t d, int32_t F)
{
    return check_glu(T, d, F, TWELL_BF16, TWELL_ACT_RELU) == TWELL_OK ? twell::glu_forward_most_ws(T, d, F, TWELL_BF16, true)
                                                                      : 0;
}

int twell_glu_forward_packed(const void *x, const void *wg_t, const void *wu_t, int32_t T, int32_t d, int32_t F,
                             int32_t act, void *h, const twell_packed_t *g, const twell_packed_t *u, int32_t keep_sign,
                             void *workspace, size_t workspace_bytes, void *stream)
{
    TWELL_TRY(check_glu(T, d, F, TWELL_BF16, act));
    if (T == 0)
        return TWELL_OK;
    for (const void *p : {x, wg_t, wu_t, (const void *)h})
        TWELL_TRY(check_mat(p));
    TWELL_TRY(check_packed(g, 16));
    TWELL_TRY(check_packed(u, 16));
    TWELL_TRY(check_ws(workspace, workspace_bytes, twell::glu_forward_ws(T, d, F, TWELL_BF16, true)));
    twell::GluFwd a{};
    a.T = T;
    a.d = d;
    a.F = F;
    a.act = act;
    a.x = x;
    a.wg = wg_t;
    a.wu = wu_t;
    a.h = h;
    a.g8 = packed8(g);
    a.u8 = packed8(u);
    a.keep_sign = keep_sign != 0;
    a.part = static_cast<float *>(workspace);
    return hip_status(twell::launch_glu(TWELL_BF16, a, static_cast<hipStream_t>(stream)));
}

int twell_glu_backward_packed(const void *x, const void *wg_t, const void *wu_t, const twell_packed_t *g,
                              const twell_packed_t *u, const void *dh, int32_t T, int32_t d, int32_t F, int32_t act,
                              void *h, void *dx, void *dwg, void *dwu, void *workspace, size_t workspace_bytes,
                              void *stream)
{
    TWELL_TRY(check_glu(T, d, F, TWELL_BF16, act));
    if (T > 0) {
        for (const void *p : {x, wg_t, wu_t, dh})
            TWELL_TRY(check_mat(p));
        TWELL_TRY(check_packed(g, 16));
        TWELL_TRY(check_packed(u, 16));
        if (!dx && !dwg && !h)
            return TWELL_E_NULL;
    }
    if (!dwg != !dwu)
        return TWELL_E_NULL;
    if (!aligned16(dx) || !aligned16(dwg) || !aligned16(dwu) || !aligned16(h))
        return TWELL_E_ALIGN;
    const twell::GluWs w = twell::glu_backward_ws(T, d, F, TWELL_BF16);
    TWELL_TRY(check_ws(workspace, workspace_bytes, w.bytes));
    twell::GluBwd a{};
    a.T = T;
    a.d = d;
    a.F = F;
    a.act = act;
    a.x = x;
    a.wg = wg_t;
    a.wu = wu_t;
    a.dh = dh;
    if (T > 0) {
        a.g8 = packed8(g);
        a.u8 = packed8(u);
    }
    a.h = h;
    a.dx = dx;
    a.dwg = dwg;
    a.dwu = dwu;
    a.dgu = workspace;
    a.ws = w;
    return hip_status(twell::launch_glu_backward(TWELL_BF16, a, static_cast<hipStream_t>(stream)));
}

int twell_act_pack(const void *x, int32_t T, int32_t d, int32_t vdtype, const twell_packed_t *to, void *stream)
{
    TWELL_TRY(check_act(T, d, vdtype));
    if (T == 0)
        return TWELL_OK;
    TWELL_TRY(check_vec(x, elem_size(vdtype)));
    TWELL_TRY(check_packed(to, 1));
    if (packed_overlaps(to, x, T, d, vdtype))
        return TWELL_E_SHAPE;
    return hip_status(twell::launch_act_pack(vdtype, x, T, d, packed8(to), static_cast<hipStream_t>(stream)));
}

int twell_act_unpack(const twell_packed_t *from, int32_t T, int32_t d, int32_t vdtype, void *out, void *stream)
{
    TWELL_TRY(check_act(T, d, vdtype));
    if (T == 0)
        return TWELL_OK;
    TWELL_TRY(check_packed(from, 1));
    TWELL_TRY(check_vec(out, elem_size(vdtype)));
    if (packed_overlaps(from, out, T, d, vdtype))
        return TWELL_E_SHAPE;
    return hip_status(twell::launch_act_unpack(vdtype, packed8(from), T, d, out, static_cast<hipStream_t>(stream)));
}

int twell_block_norm_forward(const twell_block_norm_t *bn, const void *res, const void *y, void *out, void *n,
                             void *stream)
{
    TWELL_TRY(check_block_norm(bn, bn && y && bn->gate_span));
    if (bn->T == 0)
        return TWELL_OK;
    const int rs = elem_size(bn->rdtype);
    TWELL_TRY(check_vec(res, rs));
    if (y)
        TWELL_TRY(check_vec(y, elem_size(bn->ydtype)));
    else
        out = nullptr;
    if (!out && !n)
        return TWELL_E_NULL;
    if (out)
        TWELL_TRY(check_vec(out, rs));
    if (n)
        TWELL_TRY(check_vec(n, elem_size(bn->ndtype)));
    twell::BnArgs a = bn_args(bn, y != nullptr);
    a.res = bn_tensor(res, bn->rdtype);
    a.y = bn_tensor(y, bn->ydtype);
    a.out = bn_tensor(out, bn->rdtype);
    a.n = bn_tensor(n, bn->ndtype);
    return hip_status(twell::launch_block_norm(a, bn->kind == TWELL_NORM_LAYER, bn_wide(a),
                                               static_cast<hipStream_t>(stream)));
}

size_t twell_block_norm_workspace_bytes(int32_t T, int32_t d)
{
    if (T < 0 || T > MOST_ROWS || d < 1 || d > twell::BN_MAX_D)
        return 0;
    return twell::block_norm_ws(twell::block_norm_most_groups(T, d), d);
}

int twell_block_norm_backward(const twell_block_norm_t *bn, const void *out, const void *y, const void *dout,
                              const void *dn, int32_t dndtype, void *dres, void *dy, void *dgate, float *dw_post,
                              float *db_post, float *dw_pre, float *db_pre, void *workspace, size_t workspace_bytes,
                              void *stream)
{
    const bool gated = bn && y && bn->gate_span;
    TWELL_TRY(check_block_norm(bn, gated));
    if (!known_dtype(dndtype))
        return TWELL_E_UNSUPPORTED;
    const int rs = elem_size(bn->rdtype), ys = elem_size(bn->ydtype);
    for (const float *w : {dw_post, db_post, dw_pre, db_pre})
        if (w)
            TWELL_TRY(check_vec(w, 4));
    if (bn->T > 0) {
        if (!dout && !dn)
            return TWELL_E_NULL;
        if (dout)
            TWELL_TRY(check_vec(dout, rs));
        if (dn) {
            TWELL_TRY(check_vec(dn, elem_size(dndtype)));
            TWELL_TRY(check_vec(out, rs));
        }
        TWELL_TRY(check_vec(dres, rs));
        if (y) {
            TWELL_TRY(check_vec(y, ys));
            TWELL_TRY(check_vec(dy, ys));
        }
        if (gated)
            TWELL_TRY(check_vec(dgate, rs));
        TWELL_TRY(check_ws(workspace, workspace_bytes,
                           twell::block_norm_ws(twell::block_norm_groups(bn->T, bn->d), bn->d)));
    }
    twell::BnArgs a = bn_args(bn, y != nullptr);
    a.res = bn_tensor(dn ? out : nullptr, bn->rdtype);
    a.y = bn_tensor(y, bn->ydtype);
    a.dout = bn_tensor(dout, bn->rdtype);
    a.dn = bn_tensor(dn, dndtype);
    a.dres = bn_tensor(dres, bn->rdtype);
    a.dy = bn_tensor(dy, bn->ydtype);
    a.dgate = bn_tensor(gated ? dgate : nullptr, bn->rdtype);
    a.dw[0] = dw_post;
    a.dw[1] = db_post;
    a.dw[2] = dw_pre;
    a.dw[3] = db_pre;
    a.part = static_cast<float *>(workspace);
    a.groups = twell::block_norm_groups(bn->T, bn->d);
    a.rows = twell::block_norm_rows(bn->T, bn->d);
    return hip_status(twell::launch_block_norm_backward(a, bn->kind == TWELL_NORM_LAYER, bn_wide(a),
                                                        static_cast<hipStream_t>(stream)));
}

int twell_adamw_step(const twell_adamw_tensor_t *tensors, int32_t count, int32_t state_bits, double lr, double beta1,
                     double beta2, double eps, int64_t step, uint32_t seed, const float *grad_scale, void *stream)
{
    // (eps as the kernel has it: in 32 bits)
    if (count < 0 || step < 1 || !(lr >= 0) || !(beta1 >= 0 && beta1 < 1) || !(beta2 >= 0 && beta2 < 1) ||
        !((float)eps > 0))
        return TWELL_E_SHAPE;
    if (state_bits != 8 && state_bits != 32)
        return TWELL_E_UNSUPPORTED;
    if (count == 0)
        return TWELL_OK;
    if (!tensors)
        return TWELL_E_NULL;
    const bool coded = state_bits == 8;
    for (int32_t i = 0; i < count; ++i)
        TWELL_TRY(check_adamw(tensors[i], coded, false));
    if (grad_scale && !aligned_to(grad_scale, 4))
        return TWELL_E_ALIGN;
    hipStream_t s = static_cast<hipStream_t>(stream);
    twell::AwBatch b{};
    b.beta1 = (float)beta1;
    b.omb1 = (float)(1 - beta1);
    b.beta2 = (float)beta2;
    b.omb2 = (float)(1 - beta2);
    b.eps = (float)eps;
    b.size = (float)(lr / (1 - std::pow(beta1, (double)step)));
    b.root = (float)(1 / std::sqrt(1 - std::pow(beta2, (double)step)));
    b.grad_scale = grad_scale;
    b.passes = aw_passes(tensors, count);
    int64_t chunks = 0;
    for (int32_t i = 0; i < count; ++i) {
        const twell_adamw_tensor_t &t = tensors[i];
        const int64_t c = aw_chunks(t.n, b.passes);
        if (c == 0)
            continue;
        if (b.count == twell::AW_BATCH || chunks + c > AW_MOST_CHUNKS) {
            TWELL_TRY(hip_status(twell::launch_adamw(b, coded, (int)chunks, s)));
            b.count = 0;
            chunks = 0;
        }
        const bool vec = aligned16(t.p) && aligned16(t.grad) && aligned16(t.copy) &&
                         aligned_to(t.m, coded ? 8 : 16) && aligned_to(t.v, coded ? 8 : 16);
        twell::AwTensor &o = b.t[b.count++];
        o.n = t.n;
        o.p = t.p;
        o.copy = static_cast<__bf16 *>(t.copy);
        o.grad = t.grad;
        o.m = t.m;
        o.v = t.v;
        o.m_scale = t.m_scale;
        o.v_scale = t.v_scale;
        o.decay = (float)(1 - lr * t.weight_decay);
        o.flags = (t.pdtype == TWELL_BF16 ? twell::AW_P_BF16 : 0) | (t.gdtype == TWELL_BF16 ? twell::AW_G_BF16 : 0) |
                  (vec ? twell::AW_VEC : 0);
        o.key = seed * 0x9E3779B9u + (uint32_t)i * 0x632BE5ABu;
        o.chunk0 = (int32_t)chunks;
        chunks += c;
    }
    return b.count ? hip_status(twell::launch_adamw(b, coded, (int)chunks, s)) : TWELL_OK;
}

int twell_adamw_unpack(const twell_adamw_tensor_t *tensors, int32_t count, void *stream)
{
    if (count < 0)
        return TWELL_E_SHAPE;
    if (count == 0)
        return TWELL_OK;
    if (!tensors)
        return TWELL_E_NULL;
    for (int32_t i = 0; i < count; ++i)
        TWELL_TRY(check_adamw(tensors[i], true, true));
    hipStream_t s = static_cast<hipStream_t>(stream);
    twell::AwUnpack b{};
    b.passes = aw_passes(tensors, count);
    int64_t chunks = 0;
    for (int32_t i = 0; i < count; ++i) {
        const twell_adamw_tensor_t &t = tensors[i];
        const int64_t c = aw_chunks(t.n, b.passes);
        if (c == 0)
            continue;
        if (b.count == twell::AW_BATCH || chunks + c > AW_MOST_CHUNKS) {
            TWELL_TRY(hip_status(twell::launch_adamw_unpack(b, (int)chunks, s)));
            b.count = 0;
            chunks = 0;
        }
        auto &o = b.t[b.count++];
        o.n = t.n;
        o.m = static_cast<const uint8_t *>(t.m);
        o.v = static_cast<const uint8_t *>(t.v);
        o.m_scale = t.m_scale;
        o.v_scale = t.v_scale;
        o.m_values = t.m_values;
        o.v_values = t.v_values;
        o.chunk0 = (int32_t)chunks;
        o.vec = aligned_to(t.m, 8) && aligned_to(t.v, 8) && aligned16(t.m_values) && aligned16(t.v_values);
        chunks += c;
    }
    return b.count ? hip_status(twell::launch_adamw_unpack(b, (int)chunks, s)) : TWELL_OK;
}

}  // extern "C"
