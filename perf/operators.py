"""The dense training and serving operators next to the sparse FFN, as measured cases.

Three operators, each as a plain form (elementary torch operations in 32 bits)
and as the calls a program makes of the library (``own``):

* ``glu``   h = act(x Wg) * (x Wu) and its backward pass
* ``norm``  a block's norms before and after it, with its gate, residual scale
            and residual sum, and their backward pass
* ``adamw`` one AdamW step over many tensors, states in 32 or in 8 bits

Weights lie as [F][d], one contiguous row of d per hidden neuron.
"""

import itertools
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
QBLOCK = 256        # elements that share a scale of the 8-bit states
M_OFF = 889         # 8-bit first moment: sign and 7 bits, 3 of mantissa, 127 = the block's largest
V_OFF = 1777        # 8-bit root of the second moment: 8 bits, 4 of mantissa, 255 = the block's largest
MASK = 0xFFFFFFFF


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one token of the 2B-like layer: generation of a single sequence
        dict(name="glu_fwd_token", op="glu_fwd", T=1, d=2048, F=8192, act="silu", dtype="bf16", save=False),
        # a ragged batch of tokens in serving, 0.5B-like layer
        dict(name="glu_fwd_batch", op="glu_fwd", T=45, d=1024, F=4096, act="gelu_tanh", dtype="bf16", save=False),
        # the small 32-bit layer that the tests use
        dict(name="glu_fwd_f32", op="glu_fwd", T=64, d=256, F=1024, act="relu", dtype="f32", save=True),
        # a training step's forward pass, 2B-like layer, g and u kept for the backward pass
        dict(name="glu_fwd_2b", op="glu_fwd", T=8192, d=2048, F=8192, act="silu", dtype="bf16", save=True),
        # a short last batch, 0.5B-like layer
        dict(name="glu_bwd_ragged", op="glu_bwd", T=1003, d=1024, F=4096, act="gelu", dtype="bf16"),
        # a training step's backward pass, 2B-like layer
        dict(name="glu_bwd_2b", op="glu_bwd", T=8192, d=2048, F=8192, act="silu", dtype="bf16"),
        # between two blocks while one token is generated
        dict(name="norm_fwd_token", op="norm_fwd", T=1, d=2048, kind="rms", post=True, pre=True, bias=False, span=0,
             stream="bf16", block="bf16", nxt="bf16"),
        # between two blocks in training: norm after, gate of d values, residual sum, norm before the next
        dict(name="norm_fwd_2b", op="norm_fwd", T=8192, d=2048, kind="rms", post=True, pre=True, bias=False,
             span=8192, stream="bf16", block="bf16", nxt="bf16"),
        # its backward pass with a 32-bit residual stream, the sparse FFN's 32-bit y and dx, one gate row a sequence
        dict(name="norm_bwd_2b", op="norm_bwd", T=8192, d=2048, kind="rms", post=True, pre=True, bias=False,
             span=2048, stream="f32", block="f32", nxt="bf16", dn="f32"),
        # layer norms with biases at an odd width, a gate value for every token and channel
        dict(name="norm_bwd_odd", op="norm_bwd", T=777, d=1001, kind="layer", post=True, pre=True, bias=True, span=1,
             stream="f32", block="f32", nxt="f32", dn="f32"),
        # one 2B-like layer's weights, 32-bit states and parameters, 16-bit copies for the layer
        dict(name="adamw_layer_2b", op="adamw", layers=1, d=2048, F=8192, bits=32, scaled=False),
        # 24 0.5B-like layers, 8-bit states, gradients scaled by a clip coefficient on the GPU; the states go on in 32
        # bits, as into a checkpoint
        dict(name="adamw_stack_8bit", op="adamw", layers=24, d=1024, F=4096, bits=8, scaled=True),
    ]


def _log(rng, lo, hi, unit=1):
    """A multiple of `unit` from lo to hi, spread over the logarithm."""
    n = round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / unit) * unit
    n = min(hi // unit * unit, max(lo, n))
    return n + unit if n == 3 << 10 else n  # a width of no model here


def draw(rng):
    op = rng.choice(("glu_fwd", "glu_bwd", "norm_fwd", "norm_bwd", "adamw"))
    if op.startswith("glu"):
        dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
        d, F = _log(rng, 64, 4096, 64), _log(rng, 64, 8192, 64)
        most = 8192 * 2048 * 8192 // (1 if dtype == "bf16" else 16)
        c = dict(op=op, T=_log(rng, 1, min(16384, most // (d * F))), d=d, F=F,
                 act=rng.choice(("relu", "silu", "gelu", "gelu_tanh")), dtype=dtype)
        return dict(c, save=rng.random() < 0.5) if op == "glu_fwd" else c
    if op.startswith("norm"):
        d = _log(rng, 16, 8192, rng.choice((8, 8, 1)))
        T = _log(rng, 1, 8192 * 2048 // d)
        post, pre = rng.choice(((True, True), (True, True), (False, True), (True, False)))
        c = dict(op=op, T=T, d=d, kind=rng.choice(("rms", "rms", "layer")), post=post, pre=pre,
                 bias=rng.random() < 0.3, span=rng.choice((0, 1, _log(rng, 1, T), T)),
                 stream=rng.choice(("bf16", "f32")), block=rng.choice(("bf16", "f32")), nxt=rng.choice(("bf16", "f32")))
        return dict(c, dn=rng.choice(("bf16", "f32"))) if op == "norm_bwd" else c
    return dict(op="adamw", count=_log(rng, 1, 128), largest=_log(rng, 256, 1 << 22), mix=rng.randrange(1 << 20),
                bits=rng.choice((8, 32)), scaled=rng.random() < 0.5)


def _sizes(case):
    """Elements of each tensor of a step, and whether it is a matrix of the layer (16-bit copy, weight decay)."""
    if "layers" in case:
        d, F = case["d"], case["F"]
        return [(n, mat) for _ in range(case["layers"])
                for n, mat in ((F * d, True), (F * d, True), (F * d, True), (d, False), (d, False))]
    rng = random.Random(case["mix"])  # the largest first, then sizes spread over the range below it
    sizes = [case["largest"]] + [_log(rng, 1, case["largest"]) for _ in range(case["count"] - 1)]
    return [(n, n >= 2048) for n in sizes]


# ---------------------------------------------------------------- the work a pass cannot do without
def work(case):
    op = case["op"]
    if op.startswith("glu"):
        T, d, F, es = case["T"], case["d"], case["F"], DT[case["dtype"]].itemsize
        if op == "glu_fwd":
            return {"bytes": es * (T * d + 2 * F * d + T * F * (3 if case["save"] else 1)), "flops": 4 * T * d * F}
        return {"bytes": es * (3 * T * F + 2 * T * d + 4 * F * d), "flops": 8 * T * d * F}
    if op.startswith("norm"):
        T, d = case["T"], case["d"]
        s, b, n = (DT[case[k]].itemsize for k in ("stream", "block", "nxt"))
        vecs = (1 + case["bias"]) * (case["post"] + case["pre"])
        gates = -(-T // case["span"]) if case["span"] else 0
        if op == "norm_fwd":
            per = 2 * s + b + (n if case["pre"] else 0)
            return {"bytes": T * d * per + d * (4 * vecs + s * gates), "flops": T * d * (4 + 4 * (case["post"] + case["pre"]))}
        per = 2 * s + 2 * b + (s + DT[case["dn"]].itemsize if case["pre"] else 0)
        return {"bytes": T * d * per + d * (8 * vecs + 2 * s * gates), "flops": T * d * (4 + 12 * (case["post"] + case["pre"]))}
    # p read and written, the gradient, the copy; the states read and written, those of 8 bits handed on in 32
    st = 16 if case["bits"] == 32 else 4 * (1 + 4 / QBLOCK) + 8
    sizes = _sizes(case)
    return {"bytes": int(sum(n * (8 + st + 4) for n, _ in sizes)), "flops": sum(15 * n for n, _ in sizes)}


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*shape, scale=1.0, shift=0.0, dtype="f32"):
        t = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
        return t.mul_(scale).add_(shift).to(DT[dtype])

    def new(*shape, dtype="f32"):
        return torch.empty(shape, device="cuda", dtype=DT[dtype])

    op = case["op"]
    st = {"op": op, "case": case}
    if op.startswith("glu"):
        T, d, F, dt = case["T"], case["d"], case["F"], case["dtype"]
        st.update(x=rnd(T, d, dtype=dt), wg=rnd(F, d, scale=d ** -0.5, dtype=dt), wu=rnd(F, d, scale=d ** -0.5, dtype=dt))
        if op == "glu_fwd":
            st.update(h=new(T, F, dtype=dt))
            if case["save"]:
                st.update(g=new(T, F, dtype=dt), u=new(T, F, dtype=dt))
        else:
            st.update(g=rnd(T, F, dtype=dt), u=rnd(T, F, dtype=dt), dh=rnd(T, F, scale=0.02, dtype=dt),
                      dx=new(T, d, dtype=dt), dwg=new(F, d, dtype=dt), dwu=new(F, d, dtype=dt))
        if own:
            import unstructured_sparse_transformer_amd as tw
            size = tw.glu_workspace if op == "glu_fwd" else tw.glu_backward_workspace
            st["ws"] = size(T, d, F, DT[dt])
    elif op.startswith("norm"):
        T, d, span = case["T"], case["d"], case["span"]
        bias = case["bias"]
        st.update(res=rnd(T, d, scale=2.0, dtype=case["stream"]), y=rnd(T, d, shift=0.1, dtype=case["block"]))
        st["gate"] = rnd(-(-T // span), d, scale=0.3, shift=0.5, dtype=case["stream"]) if span else None
        for k in ("post", "pre"):
            st["w_" + k] = rnd(d, scale=0.1, shift=1.0) if case[k] else None
            st["b_" + k] = rnd(d, scale=0.1) if case[k] and bias else None
        if op == "norm_fwd":
            st.update(out=new(T, d, dtype=case["stream"]), n=new(T, d, dtype=case["nxt"]) if case["pre"] else None)
        else:
            st.update(dout=rnd(T, d, scale=0.02, dtype=case["stream"]), dres=new(T, d, dtype=case["stream"]),
                      dn=rnd(T, d, scale=0.02, dtype=case["dn"]) if case["pre"] else None,
                      dy=new(T, d, dtype=case["block"]),
                      dgate=new(-(-T // span), d, dtype=case["stream"]) if span else None)
            for k in ("w_post", "b_post", "w_pre", "b_pre"):
                st["d" + k] = new(d) if st[k] is not None else None
        if own:
            import unstructured_sparse_transformer_amd as tw
            st["bn"] = tw.BlockNorm(kind=case["kind"], eps=1e-6, alpha=0.7, post=case["post"], w_post=st["w_post"],
                                    b_post=st["b_post"], w_pre=st["w_pre"], b_pre=st["b_pre"])
            if op == "norm_bwd":
                st["ws"] = tw.block_norm_workspace(T, d)
    else:
        # each kind of data lies in one buffer, a tensor is a slice of it that starts at a whole block
        sizes = _sizes(case)
        ends = list(itertools.accumulate(-(-n // QBLOCK) * QBLOCK for n, _ in sizes))
        total, coded = ends[-1], case["bits"] == 8
        st.update(lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-8, step=700, seed=seed & MASK, sets=[],
                  clip=torch.full((1,), 0.37, device="cuda") if case["scaled"] else None,
                  p=rnd(total, scale=0.02), copy=torch.zeros(total, device="cuda", dtype=torch.bfloat16))
        m, r = rnd(total, scale=3e-4), rnd(total, scale=5e-4).abs_().add_(1e-4)
        if coded:
            x = _mix(total, (seed * 97 + 1) & MASK, 0)
            st["m"], st["m_scale"] = _encode(m, x & 0xFFFFF, M_OFF, 20)
            st["v"], st["v_scale"] = _encode(r, x >> 13, V_OFF, 19)
            st.update(m_values=m, v_values=r)
        else:
            st.update(m=m, v=r.square_())
        for (n, mat), end, first in zip(sizes, ends, [0] + ends):
            t = dict(p=st["p"][first:first + n], grad=rnd(n, scale=1e-3, dtype="bf16" if mat else "f32"),
                     copy=st["copy"][first:first + n] if mat else None, weight_decay=0.1 if mat else 0.0,
                     m=st["m"][first:first + n], v=st["v"][first:first + n])
            if coded:
                t.update(m_scale=st["m_scale"][first // QBLOCK:end // QBLOCK],
                         v_scale=st["v_scale"][first // QBLOCK:end // QBLOCK],
                         m_values=m[first:first + n], v_values=r[first:first + n])
            st["sets"].append(t)
        if own:
            import unstructured_sparse_transformer_amd as tw
            st["handle"] = tw.AdamWTensors(st["sets"])
    return st


# ---------------------------------------------------------------- plain forms
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
    c = st["case"]
    dt = DT[c["dtype"]]
    x, wg, wu = st["x"].float(), st["wg"].float(), st["wu"].float()
    if c["op"] == "glu_fwd":
        g, u = x @ wg.t(), x @ wu.t()
        h = (_act(g, c["act"]) * u).to(dt)
        return {"h": h, "g": g.to(dt), "u": u.to(dt)} if c["save"] else {"h": h}
    g, u, dh = st["g"].float(), st["u"].float(), st["dh"].float()
    dg, du = dh * u * _act_grad(g, c["act"]), dh * _act(g, c["act"])
    return {"dx": (dg @ wg + du @ wu).to(dt), "dwg": (dg.t() @ x).to(dt), "dwu": (du.t() @ x).to(dt)}


def _hat(v, kind):
    """The normalised rows and the reciprocal of their deviation."""
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    rstd = torch.rsqrt((v * v).mean(1, keepdim=True) + 1e-6)
    return v * rstd, rstd


def _affine(v, w, b):
    v = v * w
    return v if b is None else v + b


def _hat_grad(dv, hat, rstd, kind):
    out = dv - hat * (dv * hat).mean(1, keepdim=True)
    if kind == "layer":
        out = out - dv.mean(1, keepdim=True)
    return out * rstd


def _plain_norm(st):
    c, kind, alpha = st["case"], st["case"]["kind"], 0.7
    T, d, span = c["T"], c["d"], c["span"]
    res, y = st["res"].float(), st["y"].float()
    rows = torch.arange(T, device="cuda") // span if span else None
    gate = st["gate"].float()[rows] if span else None
    if c["post"]:
        yhat, yr = _hat(y, kind)
        p = _affine(yhat, st["w_post"], st["b_post"])
    else:
        p = y
    if c["op"] == "norm_fwd":
        r = res + alpha * (p * gate if span else p)
        got = {"out": r.to(DT[c["stream"]])}
        if c["pre"]:
            got["n"] = _affine(_hat(r, kind)[0], st["w_pre"], st["b_pre"]).to(DT[c["nxt"]])
        return got
    got, dr = {}, st["dout"].float()  # here res holds the forward's sum, and y its block output
    if c["pre"]:
        dn, (rhat, rr) = st["dn"].float(), _hat(res, kind)
        dr = dr + _hat_grad(dn * st["w_pre"], rhat, rr, kind)
        got["dw_pre"] = (dn * rhat).sum(0)
        if c["bias"]:
            got["db_pre"] = dn.sum(0)
    got["dres"] = dr.to(DT[c["stream"]])
    dp = alpha * dr
    if span:
        padded = torch.nn.functional.pad(dp * p, (0, 0, 0, -T % span))
        got["dgate"] = padded.view(-1, span, d).sum(1).to(DT[c["stream"]])
        dp = dp * gate
    if c["post"]:
        got["dw_post"] = (dp * yhat).sum(0)
        if c["bias"]:
            got["db_post"] = dp.sum(0)
        dp = _hat_grad(dp * st["w_post"], yhat, yr, kind)
    got["dy"] = dp.to(DT[c["block"]])
    return got


def _mix(n, seed, i):
    """32 well-mixed bits for each of n elements of tensor i."""
    key = (seed * 0x9E3779B9 + i * 0x632BE5AB) & MASK
    x = torch.arange(n, device="cuda", dtype=torch.int64)
    x = (x + (x >> 32) * 0x5851F42D + key) & MASK
    x = ((x ^ (x >> 16)) * 0xA2C1B5D3) & MASK
    x = ((x ^ (x >> 15)) * 0x6D9E3C8B) & MASK
    return x ^ (x >> 16)


def _blocks(x):
    return torch.nn.functional.pad(x, (0, -x.numel() % QBLOCK)).view(-1, QBLOCK)


def _encode(x, noise, off, shift):
    """8-bit codes of x and the scale of each block: the magnitude over the block's largest, its float bits
    rounded up or down by the noise to the mantissa that is kept."""
    a = _blocks(x.abs())
    top = a.amax(1)
    scale = torch.where(top < 1e-30, torch.zeros_like(top), top)
    inv = torch.where(top < 1e-30, torch.zeros_like(top), torch.ones_like(top) / top)
    q = (a * inv[:, None]).clamp_max(1.0).view(-1)[: x.numel()]
    code = (((q.view(torch.int32).to(torch.int64) + noise) >> shift) - off).clamp(0, 127 if shift == 20 else 255)
    if shift == 20:
        code = code + 128 * (x < 0)
    else:  # a root above 0 stays above 0: it divides
        code = torch.where(q > 0, code.clamp_min(1), code)
    return code.to(torch.uint8), scale


def _decode(code, scale, off, shift):
    """The values that 8-bit codes stand for."""
    c = code.to(torch.int32)
    mag = c & 127 if shift == 20 else c
    val = torch.where(mag > 0, (mag + off) << shift, 0).view(torch.float32)
    val = torch.where(c > 127, -val, val) if shift == 20 else val
    return (_blocks(val) * scale[:, None]).view(-1)[: code.numel()]


def _states(st):
    """What a step changes, the 8-bit states as the values that they stand for."""
    coded = "m_values" in st
    return {"p": st["p"], "copy": st["copy"], "m": st["m_values" if coded else "m"], "v": st["v_values" if coded else "v"]}


def _coefficients(st):
    b1, b2 = st["beta1"], st["beta2"]
    return b1, 1 - b1, b2, 1 - b2, st["lr"] / (1 - b1 ** st["step"]), 1 / math.sqrt(1 - b2 ** st["step"])


def _plain_adamw(st):
    b1, c1, b2, c2, size, root = _coefficients(st)
    for i, t in enumerate(st["sets"]):
        g = t["grad"].float()
        if st["clip"] is not None:
            g = g * st["clip"]
        coded = t["m"].dtype == torch.uint8
        if coded:
            r = _decode(t["v"], t["v_scale"], V_OFF, 19)
            m, v = _decode(t["m"], t["m_scale"], M_OFF, 20), r * r
        else:
            m, v = t["m"], t["v"]
        m = m * b1 + g * c1
        v = v * b2 + (g * g) * c2
        r = torch.sqrt(v)
        t["p"].copy_(t["p"] * (1 - st["lr"] * t["weight_decay"]) - (m / (r * root + st["eps"])) * size)
        if t["copy"] is not None:
            t["copy"].copy_(t["p"])
        if coded:
            x = _mix(m.numel(), st["seed"], i)
            for k, val, noise, off, shift in (("m", m, x & 0xFFFFF, M_OFF, 20), ("v", r, x >> 13, V_OFF, 19)):
                code, scale = _encode(val, noise, off, shift)
                t[k].copy_(code)
                t[k + "_scale"].copy_(scale)
                val = _decode(code, scale, off, shift)
                t[k + "_values"].copy_(val * val if k == "v" else val)
        else:
            t["m"].copy_(m)
            t["v"].copy_(v)
    return _states(st)


# ---------------------------------------------------------------- one pass
def run(st):
    c, op = st["case"], st["op"]
    if not own:
        return _plain_adamw(st) if op == "adamw" else _plain_glu(st) if op.startswith("glu") else _plain_norm(st)
    import unstructured_sparse_transformer_amd as tw
    if op == "glu_fwd":
        tw.twell_glu_forward(st["x"], st["wg"], st["wu"], c["act"], st["h"], st["ws"], g=st.get("g"), u=st.get("u"))
        return {"h": st["h"], "g": st["g"], "u": st["u"]} if c["save"] else {"h": st["h"]}
    if op == "glu_bwd":
        tw.twell_glu_backward(st["x"], st["wg"], st["wu"], st["g"], st["u"], st["dh"], c["act"], st["dx"], st["dwg"],
                              st["dwu"], st["ws"])
        return {k: st[k] for k in ("dx", "dwg", "dwu")}
    if op == "norm_fwd":
        tw.twell_block_norm_forward(st["bn"], st["res"], st["y"], st["out"], st["n"], gate=st["gate"], gate_span=c["span"])
        return {k: st[k] for k in ("out", "n") if st[k] is not None}
    if op == "norm_bwd":
        tw.twell_block_norm_backward(st["bn"], st["res"], st["y"], st["dout"], st["dn"], st["dres"], st["dy"], st["ws"],
                                     gate=st["gate"], gate_span=c["span"], dgate=st["dgate"], dw_post=st["dw_post"],
                                     db_post=st["db_post"], dw_pre=st["dw_pre"], db_pre=st["db_pre"])
        names = ("dw_pre", "db_pre", "dres", "dgate", "dw_post", "db_post", "dy")
        return {k: st[k] for k in names if st[k] is not None}
    tw.twell_adamw_step(st["handle"], st["lr"], st["beta1"], st["beta2"], st["eps"], st["step"], seed=st["seed"],
                        grad_scale=st["clip"])
    if "m_values" in st:  # a pass hands the 8-bit states on, as a checkpoint in 32 bits does
        tw.twell_adamw_unpack(st["handle"])
    return _states(st)


# ---------------------------------------------------------------- the definitions in 64 bits
def _act64(g, act):
    if act == "gelu":
        return g * torch.special.ndtr(g)
    if act == "gelu_tanh":
        return g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g.pow(3)))) / 2
    return torch.relu(g) if act == "relu" else g / (1 + torch.exp(-g))


def _norm64(v, w, b, kind):
    if kind == "layer":
        return (v - v.mean(1, keepdim=True)) / torch.sqrt(v.var(1, unbiased=False, keepdim=True) + 1e-6) * w + (0 if b is None else b)
    return v / torch.sqrt(v.pow(2).mean(1, keepdim=True) + 1e-6) * w + (0 if b is None else b)


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]

    def wide(name, grad=False):
        t = st[name]
        return None if t is None else t.double().requires_grad_(grad)

    if op == "glu_fwd":
        x, got = wide("x"), {}
        g, u = torch.matmul(x, wide("wg").T), torch.matmul(x, wide("wu").T)
        got["h"] = _act64(g, case["act"]) * u
        return dict(got, g=g, u=u) if case["save"] else got
    if op == "glu_bwd":
        g, u, x = wide("g", True), wide("u", True), wide("x")
        (_act64(g, case["act"]) * u).backward(wide("dh"))
        return {"dx": torch.matmul(g.grad, wide("wg")) + torch.matmul(u.grad, wide("wu")),
                "dwg": torch.matmul(g.grad.T, x), "dwu": torch.matmul(u.grad.T, x)}
    if op.startswith("norm"):
        grad = op == "norm_bwd"
        T, kind, span = case["T"], case["kind"], case["span"]
        res, y, gate = wide("res", grad), wide("y", grad), wide("gate", grad)
        par = {k: wide(k, grad) for k in ("w_post", "b_post", "w_pre", "b_pre")}
        p = _norm64(y, par["w_post"], par["b_post"], kind) if case["post"] else y
        p = 0.7 * (p if not span else p * gate.repeat_interleave(span, 0)[:T])
        if not grad:
            r = res + p
            return {"out": r, **({"n": _norm64(r, par["w_pre"], par["b_pre"], kind)} if case["pre"] else {})}
        dr = wide("dout")  # res holds the forward's sum: its gradient first, then that of what was added
        if case["pre"]:
            _norm64(res, par["w_pre"], par["b_pre"], kind).backward(wide("dn"))
            dr = dr + res.grad
        p.backward(dr)
        got = {"dres": dr, "dy": y.grad, **({"dgate": gate.grad} if span else {})}
        return {**got, **{"d" + k: v.grad for k, v in par.items() if v is not None}}
    got = {k: _states(st)[k].double() for k in ("p", "copy", "m", "v")}
    t0, first = st["step"], 0
    for t in st["sets"]:
        n = t["p"].numel()
        g = t["grad"].double() * (1.0 if st["clip"] is None else st["clip"].double())
        if case["bits"] == 8:
            m = _decode(t["m"], t["m_scale"], M_OFF, 20).double()
            v = _decode(t["v"], t["v_scale"], V_OFF, 19).double() ** 2
        else:
            m, v = t["m"].double(), t["v"].double()
        m, v = st["beta1"] * m + (1 - st["beta1"]) * g, st["beta2"] * v + (1 - st["beta2"]) * g ** 2
        p = t["p"].double() * (1 - st["lr"] * t["weight_decay"])
        p = p - st["lr"] * (m / (1 - st["beta1"] ** t0)) / (torch.sqrt(v / (1 - st["beta2"] ** t0)) + st["eps"])
        for k, val in (("p", p), ("m", m), ("v", v), ("copy", p if t["copy"] is not None else None)):
            if val is not None:
                got[k][first:first + n] = val
        first += -(-n // QBLOCK) * QBLOCK
    return got if case["bits"] == 32 else dict(got, m=None, v=None)  # 8-bit states are rounded by the noise
