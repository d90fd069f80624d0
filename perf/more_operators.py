"""What a language model of the library's layers needs around and inside them, as measured cases.

Three operators, each as a plain form (elementary torch operations) and as the
calls a program makes of the library (``own``):

* ``embed``   rows of a table for token ids, scaled, and the table's gradient
* ``logprob`` log probabilities of given tokens from logits, entropy and the top
              alternatives, and the logits' gradient
* ``act``     activations kept in 8 bits: packed and unpacked (``act_pack``), and
              the gated product h = act(x Wg) * (x Wu) that keeps g and u so, with
              its backward pass from them (``glu_packed``)
"""

import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
IDS = {32: torch.int32, 64: torch.int64}
BLOCK = 32     # elements that share a scale of the 8-bit activations
PAD = 0.02     # tokens without an id, where a case has such
BLANK = -1e30  # no logit: below every one that is not masked


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one token of a sequence that is being generated enters the 2B-like layers
        dict(name="embed_fwd_token", op="embed_fwd", T=1, V=131072, d=2048, table="bf16", out="bf16", ids=32, pad=False),
        # a training batch enters them: 16-bit copies of the table, 32-bit residual stream
        dict(name="embed_fwd_2b", op="embed_fwd", T=8192, V=131072, d=2048, table="bf16", out="f32", ids=64, pad=False),
        # a short last batch with padding at an odd width, added to the gradient that the head left in a shared table
        dict(name="embed_bwd_ragged", op="embed_bwd", T=1003, V=32768, d=1001, dout="bf16", dtable="f32", ids=64,
             pad=True, accumulate=True),
        # a training batch's gradient of the table
        dict(name="embed_bwd_2b", op="embed_bwd", T=8192, V=131072, d=2048, dout="f32", dtable="f32", ids=64, pad=False,
             accumulate=False),
        # the next token of one sequence: what it may be, at a temperature
        dict(name="logprob_token", op="logprob_fwd", T=1, V=131072, dtype="bf16", ids=64, scale=1.25, masked=0.0, k=20,
             pad=False),
        # a ragged batch in serving, 32-bit logits of an odd vocabulary, a grammar that forbids half of the tokens
        dict(name="logprob_batch", op="logprob_fwd", T=45, V=50001, dtype="f32", ids=64, scale=1.0, masked=0.5, k=8,
             pad=True),
        # a training batch's loss, and its gradient with an entropy term
        dict(name="logprob_fwd_batch", op="logprob_fwd", T=4096, V=131072, dtype="bf16", ids=64, scale=1.0, masked=0.0, k=0,
             pad=False),
        dict(name="logprob_bwd_batch", op="logprob_bwd", T=4096, V=131072, dtype="bf16", ids=64, scale=1.0, masked=0.0,
             entropy=True, pad=False),
        # the rows of a small 32-bit layer kept for later
        dict(name="act_pack_small", op="act_pack", T=64, d=1001, dtype="f32"),
        # the hidden activations of the 2B-like layer kept for the backward pass
        dict(name="act_pack_2b", op="act_pack", T=8192, d=8192, dtype="bf16"),
        # a short last batch through the 0.5B-like layer's gated product and back
        dict(name="glu_packed_ragged", op="glu_packed", T=1003, d=1024, F=4096, act="gelu_tanh"),
        # a training step's, 2B-like layer
        dict(name="glu_packed_2b", op="glu_packed", T=8192, d=2048, F=8192, act="silu"),
    ]


def _log(rng, lo, hi, unit=1):
    """A multiple of `unit` from lo to hi, spread over the logarithm."""
    n = round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / unit) * unit
    return min(hi // unit * unit, max(lo, n))


def draw(rng):
    op = rng.choice(("embed_fwd", "embed_bwd", "embed_bwd", "logprob_fwd", "logprob_fwd", "logprob_bwd", "act_pack",
                     "glu_packed"))
    kind = lambda: rng.choice(("bf16", "f32"))  # noqa: E731
    if op.startswith("embed"):
        d = _log(rng, 16, 4096, rng.choice((8, 8, 1)))
        T = _log(rng, 1, min(65536, 8192 * 2048 // d))
        c = dict(op=op, T=T, V=_log(rng, 256, min(262144, 131072 * 2048 // d)), d=d, ids=rng.choice((32, 64)),
                 pad=rng.random() < 0.5)
        if op == "embed_fwd":
            return dict(c, table=kind(), out=kind())
        return dict(c, dout=kind(), dtable=kind(), accumulate=rng.random() < 0.3)
    if op.startswith("logprob"):
        V = _log(rng, 512, 262144, rng.choice((64, 8, 1)))
        dtype = kind()
        c = dict(op=op, T=_log(rng, 1, min(16384, 4096 * 131072 // V // (1 if dtype == "bf16" else 2))), V=V, dtype=dtype,
                 ids=rng.choice((32, 64)), scale=rng.choice((1.0, 1.0, 0.5, 1.25)), masked=rng.choice((0.0, 0.0, 0.5, 0.99)),
                 pad=rng.random() < 0.5)
        return dict(c, k=rng.choice((0, 1, 5, 20, 64))) if op == "logprob_fwd" else dict(c, entropy=rng.random() < 0.5)
    if op == "act_pack":
        d = _log(rng, 16, 16384, rng.choice((32, 8, 1)))
        return dict(op=op, T=_log(rng, 1, 8192 * 4096 // d), d=d, dtype=kind())
    d, F = _log(rng, 64, 4096, 64), _log(rng, 64, 8192, 64)
    return dict(op=op, T=_log(rng, 1, min(16384, 8192 * 2048 * 8192 // (d * F))), d=d, F=F,
                act=rng.choice(("relu", "silu", "gelu", "gelu_tanh")))


# ---------------------------------------------------------------- the work a pass cannot do without
def _chance(V):
    """Of each id (see prepare): ln((v + 2) / (v + 1)) / ln(V + 1)."""
    v = np.arange(1, V + 1, dtype=np.float64)
    return np.log1p(1 / v) / math.log(V + 1)


def work(case):
    op, T = case["op"], case["T"]
    if op.startswith("embed"):
        V, d, idb = case["V"], case["d"], case["ids"] // 8
        rows = float((1 - (1 - _chance(V)) ** T).sum())  # that have tokens
        if op == "embed_fwd":
            return {"bytes": rows * d * DT[case["table"]].itemsize + T * (d * DT[case["out"]].itemsize + idb), "flops": T * d}
        gs = DT[case["dtable"]].itemsize
        return {"bytes": T * (d * DT[case["dout"]].itemsize + idb) + (2 * rows if case["accumulate"] else V) * d * gs,
                "flops": T * d}
    if op.startswith("logprob"):
        V, es, idb = case["V"], DT[case["dtype"]].itemsize, case["ids"] // 8
        if op == "logprob_fwd":
            return {"bytes": T * (V * es + idb + 12 + 8 * case["k"]), "flops": 6 * T * V}
        return {"bytes": T * (2 * V * es + idb + 16), "flops": 6 * T * V}
    if op == "act_pack":
        d = case["d"]
        return {"bytes": T * (2 * d * DT[case["dtype"]].itemsize + 2 * (d + 2 * -(-d // BLOCK))), "flops": 4 * T * d}
    d, F = case["d"], case["F"]
    kept = 2 * T * F * (1 + 2 / BLOCK)  # g and u, written and read
    return {"bytes": int(2 * (2 * T * d + 2 * F * d + T * F) + 2 * kept + 2 * (T * F + T * d + 2 * F * d)), "flops": 12 * T * d * F}


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, T = case["op"], case["T"]

    def rnd(*shape, scale=1.0, dtype="f32"):
        t = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
        return t.mul_(scale).to(DT[dtype])

    def uni(*shape):
        return torch.rand(shape, generator=gen, device="cuda", dtype=torch.float64)

    def new(*shape, dtype="f32"):
        return torch.empty(shape, device="cuda", dtype=DT[dtype])

    def ids(V):
        """Tokens as texts have them: the v-th most frequent about 1 / v as often as the first."""
        t = (torch.exp(uni(T) * math.log(V + 1)).floor().to(torch.int64) - 1).clamp(0, V - 1)
        if case["pad"]:
            t = torch.where(uni(T) < PAD, torch.full_like(t, -1), t)
        return t.to(IDS[case["ids"]])

    st = {"op": op, "case": case}
    if op.startswith("embed"):
        V, d = case["V"], case["d"]
        st.update(ids=ids(V), scale=math.sqrt(d))
        if op == "embed_fwd":
            st.update(table=rnd(V, d, scale=0.02, dtype=case["table"]), out=new(T, d, dtype=case["out"]))
        else:
            st.update(dout=rnd(T, d, scale=0.02, dtype=case["dout"]), dtable=rnd(V, d, scale=0.01, dtype=case["dtable"]))
            if own:
                import unstructured_sparse_transformer_amd as tw
                st["ws"] = tw.embed_workspace(T, V, d)
    elif op.startswith("logprob"):
        V = case["V"]
        z = rnd(T, V)
        z.mul_(torch.exp(uni(T, 1) * math.log(16.0)).float().mul_(0.5))  # flat and peaked rows
        if case["masked"]:
            z[torch.rand((T, V), generator=gen, device="cuda") < case["masked"]] = -math.inf
            if T > 1:
                z[T // 2] = -math.inf  # a row with nothing left
        st.update(logits=z.to(DT[case["dtype"]]), targets=ids(V))
        del z
        if op == "logprob_fwd":
            k = case["k"]
            st.update(logp=new(T), norm=new(T, 2), entropy=new(T), top_logp=new(T, k) if k else None,
                      top_idx=torch.empty((T, k), device="cuda", dtype=torch.int32) if k else None)
            if own:
                import unstructured_sparse_transformer_amd as tw
                st["ws"] = tw.logprob_workspace(T, V, k)
        else:
            got = _logprob(st, 0)
            st.update(norm=got["norm"], entropy=got["entropy"], dlogp=rnd(T, scale=1 / T),
                      dentropy=rnd(T, scale=0.1 / T) if case["entropy"] else None, dlogits=torch.empty_like(st["logits"]))
    elif op == "act_pack":
        d = case["d"]
        st.update(x=rnd(T, d, dtype=case["dtype"]), out=new(T, d, dtype=case["dtype"]))
        if own:
            import unstructured_sparse_transformer_amd as tw
            st["packed"] = tw.PackedAct.empty(T, d)
    else:
        d, F = case["d"], case["F"]
        st.update(x=rnd(T, d, dtype="bf16"), wg=rnd(F, d, scale=d ** -0.5, dtype="bf16"), wu=rnd(F, d, scale=d ** -0.5, dtype="bf16"),
                  dh=rnd(T, F, scale=0.02, dtype="bf16"), h=new(T, F, dtype="bf16"), dx=new(T, d, dtype="bf16"),
                  dwg=new(F, d, dtype="bf16"), dwu=new(F, d, dtype="bf16"))
        if own:
            import unstructured_sparse_transformer_amd as tw
            st.update(g=tw.PackedAct.empty(T, F), u=tw.PackedAct.empty(T, F), ws=tw.glu_packed_workspace(T, d, F),
                      ws_backward=tw.glu_backward_workspace(T, d, F, torch.bfloat16))
    return st


# ---------------------------------------------------------------- plain forms
def _plain_embed(st):
    c = st["case"]
    ids = st["ids"].long()
    there = (ids >= 0) & (ids < c["V"])
    if c["op"] == "embed_fwd":
        rows = st["table"][ids.clamp(0, c["V"] - 1)].float() * st["scale"]
        return {"out": (rows * there[:, None]).to(DT[c["out"]])}
    total = torch.zeros((c["V"], c["d"]), device="cuda")
    total.index_add_(0, ids.clamp(0, c["V"] - 1), st["dout"].float() * there[:, None])
    total *= st["scale"]
    if c["accumulate"]:
        total += st["dtable"].float()
    st["dtable"].copy_(total)
    return {"dtable": st["dtable"]}


def _masked(z):
    """The values with a finite one in the place of -inf, and where that is."""
    none = z == -math.inf
    return z.masked_fill(none, BLANK), none


def _logprob(st, k):
    c = st["case"]
    z, none = _masked(st["logits"].float())
    top = z.amax(1, keepdim=True)
    z -= top
    z *= c["scale"]
    e = torch.exp(z).masked_fill_(none, 0)
    total, weighted = e.sum(1), z.masked_fill_(none, 0).mul_(e).sum(1)
    del z, e
    empty = none.all(1)
    size = torch.log(total).masked_fill_(empty, 0)
    got = {"norm": torch.stack((top[:, 0].masked_fill(empty, -math.inf), size), 1),
           "entropy": (size - weighted / total).masked_fill(empty, 0)}
    at = st["targets"].long()
    there = (at >= 0) & (at < c["V"])
    at = at.clamp(0, c["V"] - 1)[:, None]
    logp = (st["logits"].gather(1, at).float() - top)[:, 0] * c["scale"] - size
    got["logp"] = logp.masked_fill(empty, -math.inf).masked_fill(~there, 0)
    if k:
        # the value's bits in an order of whole numbers, then the index, lowest first
        b = st["logits"].float().view(torch.int32).to(torch.int64)
        b = torch.where(b < 0, -(b & 0x7FFFFFFF), b)
        idx = torch.arange(c["V"], device="cuda")
        got["top_idx"] = torch.topk((b << 32) - idx, k, dim=1).indices.to(torch.int32)
        val = st["logits"].gather(1, got["top_idx"].long()).float() - top
        got["top_logp"] = (val * c["scale"] - size[:, None]).masked_fill(empty[:, None], -math.inf)
    return got


def _plain_logprob_bwd(st):
    c = st["case"]
    z, none = _masked(st["logits"].float())
    top, size = st["norm"].unbind(1)
    empty = top == -math.inf
    logp = (z - top.masked_fill(empty, 0)[:, None]) * c["scale"] - size[:, None]
    p = torch.exp(logp).masked_fill_(none, 0)
    at = st["targets"].long()
    there = (at >= 0) & (at < c["V"]) & ~empty
    dlogp = st["dlogp"] * there
    dz = p * -dlogp[:, None]
    if c["entropy"]:
        dz -= p * (logp + st["entropy"][:, None]).masked_fill_(none, 0) * st["dentropy"][:, None]
    dz.scatter_add_(1, at.clamp(0, c["V"] - 1)[:, None], dlogp[:, None])
    return {"dlogits": (dz * c["scale"]).to(DT[c["dtype"]])}


def _kept(x):
    """The values that 8-bit codes of the rows stand for, in 32 bits."""
    T, d = x.shape
    v = torch.nn.functional.pad(x, (0, -d % BLOCK)).view(T, -1, BLOCK)
    top = v.abs().amax(2, keepdim=True)
    scale = top / 127
    scale = ((scale.view(torch.int32) + 0xFFFF) & -0x10000).view(torch.float32)  # up to 16 bits
    inv = torch.where(top < 1e-30, torch.zeros_like(top), 1 / scale)
    code = torch.round(v * inv).to(torch.int8)
    return (code.float() * scale).view(T, -1)[:, :d]


def _act(g, act):
    if act == "relu":
        return g.clamp_min(0)
    if act == "silu":
        return g * torch.sigmoid(g)
    if act == "gelu":
        return 0.5 * g * (1 + torch.erf(g * math.sqrt(0.5)))
    return g * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g))


def _act_grad(g, act):
    if act == "relu":
        return (g > 0).float()
    if act == "silu":
        s = torch.sigmoid(g)
        return s * (1 + g * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(g * math.sqrt(0.5))) + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))
    c = 2 * math.sqrt(2 / math.pi)
    s = torch.sigmoid(c * (g + 0.044715 * g * g * g))
    return s + g * s * (1 - s) * c * (1 + 3 * 0.044715 * g * g)


def _plain_glu(st):
    act = st["case"]["act"]
    x, wg, wu, dh = (st[k].float() for k in ("x", "wg", "wu", "dh"))
    g, u = x @ wg.t(), x @ wu.t()
    h = (_act(g, act) * u).bfloat16()
    g, u = _kept(g), _kept(u)
    dg, du = dh * u * _act_grad(g, act), dh * _act(g, act)
    grads = {"dx": dg @ wg + du @ wu, "dwg": dg.t() @ x, "dwu": du.t() @ x}
    return {"h": h, **{k: v.bfloat16() for k, v in grads.items()}}


# ---------------------------------------------------------------- one pass
def run(st):
    c, op = st["case"], st["op"]
    if not own:
        if op.startswith("embed"):
            return _plain_embed(st)
        if op == "logprob_fwd":
            return _logprob(st, c["k"])
        if op == "logprob_bwd":
            return _plain_logprob_bwd(st)
        return {"out": _kept(st["x"].float()).to(DT[c["dtype"]])} if op == "act_pack" else _plain_glu(st)
    import unstructured_sparse_transformer_amd as tw
    if op == "embed_fwd":
        tw.twell_embed_forward(st["ids"], st["table"], st["out"], scale=st["scale"])
        return {"out": st["out"]}
    if op == "embed_bwd":
        tw.twell_embed_backward(st["ids"], st["dout"], st["dtable"], st["ws"], scale=st["scale"], accumulate=c["accumulate"])
        return {"dtable": st["dtable"]}
    if op == "logprob_fwd":
        tw.twell_logprob_forward(st["logits"], st["targets"], st["logp"], st["norm"], st["ws"], scale=c["scale"],
                                 entropy=st["entropy"], top_logp=st["top_logp"], top_idx=st["top_idx"])
        return {k: st[k] for k in ("norm", "entropy", "logp", "top_idx", "top_logp") if st[k] is not None}
    if op == "logprob_bwd":
        tw.twell_logprob_backward(st["logits"], st["targets"], st["norm"], st["dlogp"], st["dlogits"], scale=c["scale"],
                                  entropy=st["entropy"], dentropy=st["dentropy"])
        return {"dlogits": st["dlogits"]}
    if op == "act_pack":
        tw.twell_act_pack(st["x"], st["packed"])
        tw.twell_act_unpack(st["packed"], st["out"])
        return {"out": st["out"]}
    tw.twell_glu_forward_packed(st["x"], st["wg"], st["wu"], c["act"], st["h"], st["g"], st["u"], st["ws"])
    tw.twell_glu_backward_packed(st["x"], st["wg"], st["wu"], st["g"], st["u"], st["dh"], c["act"], st["dx"], st["dwg"],
                                 st["dwu"], st["ws_backward"])
    return {k: st[k] for k in ("h", "dx", "dwg", "dwu")}


# ---------------------------------------------------------------- the definitions in 64 bits
def _kept64(v):
    """Each block's largest magnitude becomes 127 steps, a step held in 8 bits of mantissa, rounded up."""
    got = torch.empty_like(v)
    for first in range(0, v.shape[1], BLOCK):
        b = v[:, first:first + BLOCK]
        step = (b.abs().max(1, keepdim=True).values / 127).clamp_min(1e-300)
        unit = torch.exp2(torch.floor(torch.log2(step)) - 7)
        step = torch.ceil(step / unit) * unit
        got[:, first:first + BLOCK] = torch.round(b / step) * step
    return got


def _act64(g, act):
    if act == "gelu":
        return g * torch.special.ndtr(g)
    if act == "gelu_tanh":
        return g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g.pow(3)))) / 2
    return torch.relu(g) if act == "relu" else g / (1 + torch.exp(-g))


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op == "embed_fwd":
        wide = torch.cat((st["table"].double() * st["scale"], torch.zeros((1, case["d"]), device="cuda", dtype=torch.float64)))
        return {"out": torch.index_select(wide, 0, st["ids"].long())} if not case["pad"] else {
            "out": torch.index_select(wide, 0, torch.where(st["ids"] < 0, case["V"], st["ids"]).long())}
    if op == "embed_bwd":
        keep = st["ids"] >= 0
        start = st["dtable"].double() if case["accumulate"] else torch.zeros_like(st["dtable"], dtype=torch.float64)
        return {"dtable": torch.index_add(start, 0, st["ids"][keep].long(), st["dout"][keep].double(), alpha=st["scale"])}
    if op.startswith("logprob"):
        z = st["logits"].double() * case["scale"]
        lse = torch.logsumexp(z, 1, keepdim=True)
        empty = (lse == -math.inf)
        logp = z - torch.where(empty, torch.zeros_like(lse), lse)
        del z
        p = torch.exp(logp)
        entropy = -torch.nan_to_num(logp, neginf=0.0).mul_(p).sum(1, keepdim=True)
        given = st["targets"] >= 0
        at = torch.where(given, st["targets"], 0).long()[:, None]
        if op == "logprob_fwd":
            top = st["logits"].double().amax(1)
            size = torch.where(empty[:, 0], 0.0, lse[:, 0] - top * case["scale"])
            got = {"norm": torch.stack((top, size), 1), "entropy": entropy[:, 0].clone(), "logp": torch.where(given, logp.gather(1, at)[:, 0], 0.0)}
            if case["k"]:  # the indices are whole numbers: the values at the largest ones, whichever of equal ones they are
                got.update(top_idx=None, top_logp=torch.topk(logp, case["k"], dim=1).values)
            return got
        dlogp = torch.where(given[:, None] & ~empty, st["dlogp"].double()[:, None], 0.0)
        dz = torch.zeros_like(p).scatter_(1, at, 1.0).sub_(p).mul_(dlogp)
        if case["entropy"]:
            dz -= torch.nan_to_num(logp, neginf=0.0).add_(entropy).mul_(p).mul_(st["dentropy"].double()[:, None])
        return {"dlogits": dz.mul_(case["scale"])}
    if op == "act_pack":
        return {"out": _kept64(st["x"].double())}
    x, wg, wu, dh = (st[k].double() for k in ("x", "wg", "wu", "dh"))
    g, u = torch.matmul(x, wg.T), torch.matmul(x, wu.T)
    got = {"h": _act64(g, case["act"]) * u}
    g, u = _kept64(g).requires_grad_(), _kept64(u).requires_grad_()
    (_act64(g, case["act"]) * u).backward(dh)
    return {**got, "dx": torch.matmul(g.grad, wg) + torch.matmul(u.grad, wu), "dwg": torch.matmul(g.grad.T, x),
            "dwu": torch.matmul(u.grad.T, x)}
