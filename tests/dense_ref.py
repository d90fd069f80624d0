"""The dense layer's operators in 64 bits, from their formulas, with bounds of
what the same formulas in 32 bits may be off by (torch on any device).

u = 2^-24 is the rounding of one fp32 operation.  Every bound is a constant
number of roundings times the sum of the magnitudes of the terms that were
added, carried through the formulas to first order."""

import math

import torch

U = 2.0 ** -24
# roundings that a value of the norms may pass one after another: a row's sums (8 + 6 + 4 levels), a workgroup's
# rows and the workgroups' sums (at most 20 + 64 + 8 for the tests' T), the formulas themselves
CN = 256.0


def half_step(x, dtype):
    """Rounding a value to its storage type."""
    return x.abs() * (2.0 ** -8 if dtype == torch.bfloat16 else U)


def check(got, want, bound, label):
    got = got.double()
    bound = bound + half_step(want, got.dtype) + 1e-38
    assert got.shape == want.shape, label
    assert torch.isfinite(got).all(), f"{label}: not finite"
    off = (got - want).abs()
    assert (off <= bound).all(), f"{label}: off by {float((off / bound).max()):.3g} bounds"


# ---------------------------------------------------------------- block norms
class Norm:
    """One norm of rows v (with bound e of their error): hat, rstd and the bound of hat's error."""

    def __init__(self, v, e, kind, eps):
        c = v - v.mean(1, keepdim=True) if kind == "layer" else v
        self.rstd = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + eps)
        self.hat, self.kind = c * self.rstd, kind
        err = e.amax(1, keepdim=True) + CN * U * v.abs().amax(1, keepdim=True)  # of a centred value
        self.e = self.rstd * err * (2 + self.hat.abs())  # of hat: its value, and its share of rstd's error
        self.rel = self.rstd * err  # of rstd

    def affine(self, w, b):
        y = self.hat * w + b
        return y, self.e * w.abs() + CN * U * (self.hat * w).abs() + CN * U * b.abs()

    def back(self, g):
        out = g - self.hat * (g * self.hat).mean(1, keepdim=True)
        return self.rstd * (out - g.mean(1, keepdim=True) if self.kind == "layer" else out)

    def back_bound(self, g, e):
        """Of back(g) when g is off by e."""
        h, mean = self.hat.abs(), lambda x: x.mean(1, keepdim=True)
        terms = lambda x: x + h * mean(x * h) + (mean(x) if self.kind == "layer" else 0)  # noqa: E731
        moved = self.e * mean(g.abs() * h) + h * mean(g.abs() * self.e)
        return self.rstd * (terms(e) + moved + (CN * U + self.rel) * terms(g.abs()))


def _par(p, like):
    w, b = (None if x is None else x.double() for x in p)
    one = torch.ones(like.shape[1], dtype=torch.float64, device=like.device)
    return one if w is None else w, torch.zeros_like(one) if b is None else b


def norm_forward(res, y, gate, span, kind, eps, alpha, post, par_post, par_pre):
    """{name: (value, bound)} of out and n; par_* = (w, b)."""
    res = res.double()
    r, e = res, torch.zeros_like(res)
    if y is not None:
        y = y.double()
        p, ep = y, torch.zeros_like(y)
        if post:
            p, ep = Norm(y, ep, kind, eps).affine(*_par(par_post, y))
        g = torch.ones_like(p) if gate is None else gate.double().repeat_interleave(span, 0)[: y.shape[0]]
        r = res + alpha * g * p
        e = abs(alpha) * g.abs() * ep + CN * U * (res.abs() + (alpha * g * p).abs())
    n, en = Norm(r, e, kind, eps).affine(*_par(par_pre, r))
    return {"out": (r, e), "n": (n, en)}


def norm_backward(out, y, gate, span, dout, dn, kind, eps, alpha, post, par_post, par_pre):
    """{name: (value, bound)} of every gradient; out is taken as it is stored."""
    like = out if out is not None else dout
    got, T = {}, like.shape[0]
    dr = torch.zeros(like.shape, dtype=torch.float64, device=like.device) if dout is None else dout.double()
    e = CN * U * dr.abs()
    if dn is not None:
        v, dn = out.double(), dn.double()
        norm, (w, _) = Norm(v, torch.zeros_like(v), kind, eps), _par(par_pre, v)
        dr = dr + norm.back(dn * w)
        e = e + norm.back_bound(dn * w, CN * U * (dn * w).abs())
        got["dw_pre"] = (dn * norm.hat).sum(0), (dn.abs() * (norm.e + CN * U * norm.hat.abs())).sum(0)
        got["db_pre"] = dn.sum(0), CN * U * dn.abs().sum(0)
    got["dres"] = dr, e
    if y is None:
        return got
    y = y.double()
    p, ep = y, torch.zeros_like(y)
    norm = None
    if post:
        norm, (w, b) = Norm(y, ep, kind, eps), _par(par_post, y)
        p, ep = norm.affine(w, b)
    dp, edp = alpha * dr, abs(alpha) * e + CN * U * (alpha * dr).abs()
    if gate is not None:
        G = gate.shape[0]
        rows = torch.arange(T, device=y.device) // span
        zero = torch.zeros((G, y.shape[1]), dtype=torch.float64, device=y.device)
        got["dgate"] = (zero.index_add(0, rows, dp * p),
                        zero.index_add(0, rows, edp * p.abs() + dp.abs() * ep + CN * U * (dp * p).abs()))
        g = gate.double()[rows]
        dp, edp = dp * g, edp * g.abs() + CN * U * (dp * g).abs()
    if post:
        got["dw_post"] = (dp * norm.hat).sum(0), (edp * norm.hat.abs() + dp.abs() * norm.e
                                                  + CN * U * (dp * norm.hat).abs()).sum(0)
        got["db_post"] = dp.sum(0), (edp + CN * U * dp.abs()).sum(0)
        got["dy"] = norm.back(dp * w), norm.back_bound(dp * w, edp * w.abs() + CN * U * (dp * w).abs())
    else:
        got["dy"] = dp, edp
    return got


# ---------------------------------------------------------------- gated product
def act(g, name):
    if name == "relu":
        return g.clamp_min(0)
    if name == "silu":
        return g / (1 + torch.exp(-g))
    if name == "gelu":
        return g * 0.5 * torch.erfc(-g / math.sqrt(2))
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))


def act_grad(g, name):
    if name == "relu":
        return (g > 0).to(g.dtype)
    if name == "silu":
        s = 1 / (1 + torch.exp(-g))
        return s + g * s * (1 - s)
    if name == "gelu":
        return 0.5 * torch.erfc(-g / math.sqrt(2)) + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def glu_forward(x, wg, wu, name):
    """{name: (value, bound)} of g, u and h; an fp32 sum of K products is off by at most K u of their magnitudes."""
    x, wg, wu = x.double(), wg.double(), wu.double()
    g, u = x @ wg.T, x @ wu.T
    k = x.shape[1] * U
    eg, eu = k * (x.abs() @ wg.abs().T), k * (x.abs() @ wu.abs().T)
    a = act(g, name)
    # the activations' own 32-bit evaluation, and slopes of at most 1.13
    ea = 1.13 * eg + 4e-6 * (1 + g.abs())
    return {"g": (g, eg), "u": (u, eu), "h": (a * u, ea * u.abs() + a.abs() * eu + ea * eu)}


def glu_backward(x, wg, wu, g, u, dh, name, dtype):
    """{name: (value, bound)} of dx, dwg, dwu; dg and du are rounded to dtype before the products."""
    x, wg, wu, g, u, dh = (t.double() for t in (x, wg, wu, g, u, dh))
    dg, du = dh * u * act_grad(g, name), dh * act(g, name)
    slack = 4e-6 * (1 + g.abs()) ** 2
    eg = half_step(dg, dtype) * 1.01 + slack * (dh * u).abs()
    eu = half_step(du, dtype) * 1.01 + slack * dh.abs()
    k, t = 2 * wg.shape[0] * U, x.shape[0] * U
    ag, au = dg.abs() + eg, du.abs() + eu
    return {"dx": (dg @ wg + du @ wu, eg @ wg.abs() + eu @ wu.abs() + k * (ag @ wg.abs() + au @ wu.abs())),
            "dwg": (dg.T @ x, eg.T @ x.abs() + t * (ag.T @ x.abs())),
            "dwu": (du.T @ x, eu.T @ x.abs() + t * (au.T @ x.abs()))}
