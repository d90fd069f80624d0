"""The operators at a model's two ends and the 8-bit activations in 64 bits, from
their formulas, with bounds of what the same formulas in 32 bits may be off by
(torch on any device).

u = 2^-24 is the rounding of one fp32 operation.  Bounds count the roundings a
term may pass, times the sum of the terms' magnitudes, to first order."""

import math

import torch

from dense_ref import U, half_step

BLOCK = 32


def check(got, value, bound, label):
    """`got` within the bound of the value, and half a step of its type for the rounding to it; equal where the value is
    infinite."""
    fin = torch.isfinite(value)
    most = (bound + half_step(value.abs() + bound, got.dtype) + 1e-38)[fin]
    got = got.double()
    assert got.shape == value.shape, label
    assert torch.equal(got[~fin], value[~fin]), label
    assert torch.isfinite(got[fin]).all(), f"{label}: not finite"
    off = (got[fin] - value[fin]).abs()
    assert (off <= most).all(), f"{label}: off by {float((off / most).max()):.3g} bounds"


# ---------------------------------------------------------------- embedding
def _there(ids, V):
    ids = ids.long()
    ok = (ids >= 0) & (ids < V)
    return ids.clamp(0, V - 1), ok


def embed_forward(ids, table, scale):
    at, ok = _there(ids, table.shape[0])
    rows = table[at].double() * float(torch.tensor(scale, dtype=torch.float32)) * ok[:, None]
    return rows, U * rows.abs()


def embed_backward(ids, dout, V, scale, old=None):
    """A sum of n terms in any order is off by at most n u of their magnitudes; the scale, and the addition to what was
    there, are two roundings more.  (On the host, where a sum over one id for all tokens is quick.)"""
    device, ids, dout = dout.device, ids.cpu(), dout.cpu()
    at, ok = _there(ids, V)
    at, rows = at[ok], dout[ok].double()
    scale = float(torch.tensor(scale, dtype=torch.float32))
    zero = torch.zeros((V, dout.shape[1]), dtype=torch.float64)
    total = (zero.index_add(0, at, rows) * scale).to(device)
    size = (zero.index_add(0, at, rows.abs()) * abs(scale)).to(device)
    n = torch.zeros(V, dtype=torch.float64).index_add(0, at, torch.ones_like(at, dtype=torch.float64)).to(device)
    bound = (n[:, None] + 3) * U * size
    if old is None:
        return total, bound
    old = old.double()
    return total + old, bound + U * (old.abs() + size) * (n[:, None] > 0)


# ---------------------------------------------------------------- log probabilities
def logprob_forward(logits, targets, scale, k=0):
    """{name: (value, bound)} of norm, entropy, logp and top_logp, and the order top_idx has to have.

    x = (z - m) c in base 2 has a difference, a product, and a c of two roundings: 4 u |x|, 5 with higher orders.  exp2 is
    within 2 u: e is off by (3 + 4 |x|) u of itself.  A thread adds V / 256 terms, then 6 + 4 + 64 partial sums at most
    are joined; a larger maximum scales the sums (4 u, and 4 u of the range that it is raised by: all of these together
    are the row's range R), at most V / 1024 + 74 times."""
    z = logits.double()
    T, V = z.shape
    ln2 = math.log(2)
    m = z.amax(1, keepdim=True)
    empty = m == -math.inf
    x = torch.where(empty, 0.0, (z - m)) * scale / ln2  # -inf stays
    e = torch.where(empty | (z == -math.inf), 0.0, torch.exp2(x))
    ax = torch.where(z == -math.inf, 0.0, x).abs()
    S, W = e.sum(1), (e * ax).sum(1)
    L = torch.where(empty[:, 0], 0.0, torch.log(S))
    mean = torch.where(empty[:, 0], 0.0, W / S)  # of -x
    K = V / 128 + 8 * ax.amax(1).clamp_max(200) + 450
    eL = K * U + 4 * U * (1 + L.abs())
    eH = eL + ln2 * mean * (2 * K + 30) * U + 4 * U * (L.abs() + mean)
    got = {"norm": (torch.stack((m[:, 0], L), 1), torch.stack((torch.zeros_like(eL), eL), 1)),
           "entropy": (torch.where(empty[:, 0], 0.0, L + ln2 * mean), eH)}
    logp = torch.where(empty, -math.inf, x * ln2 - L[:, None])
    ep = 5 * U * ax * ln2 + eL[:, None] + 3 * U * torch.where(logp == -math.inf, 0.0, logp).abs()
    if targets is not None:
        at, ok = _there(targets, V)
        at = at[:, None]
        got["logp"] = torch.where(ok, logp.gather(1, at)[:, 0], 0.0), torch.where(ok, ep.gather(1, at)[:, 0], 0.0)
    idx = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]
    got["top_logp"] = logp.gather(1, idx), ep.gather(1, idx)
    return got, idx


def logprob_backward(logits, targets, norm, dlogp, scale, entropy=None, dentropy=None):
    """(value, bound) of dlogits for the stored norm and entropy.  The exponent l, in base 2, has the 5 u |x| of the
    forward pass and 4 u of the stored L; p is off by ln 2 times that and by 2 u.  A p below 2^-126 may be 0: with it goes
    at most p (|d| + |h| (|log p| + H)), and p |log p| is largest at 2^-126, where |log p| is below 88."""
    z, ln2 = logits.double(), math.log(2)
    T, V = z.shape
    m, L = norm.double().unbind(1)
    empty = (m == -math.inf)[:, None]
    x = torch.where(empty, -math.inf, z - torch.where(empty, 0.0, m[:, None])) * scale
    logp = x - L[:, None]
    p = torch.exp(logp)
    fin = torch.where(logp == -math.inf, 0.0, logp)
    ax = torch.where(x == -math.inf, 0.0, x).abs() / ln2
    q = U * (5 * ax + 4 * L.abs()[:, None] / ln2 + 2 * fin.abs() / ln2 + 4)
    dz, size = torch.zeros_like(z), torch.zeros_like(z)
    bound, lost = torch.zeros_like(z), torch.zeros((T, 1), dtype=torch.float64, device=z.device)
    if dlogp is not None:
        at, ok = _there(targets, V)
        d = torch.where(ok[:, None] & ~empty, dlogp.double()[:, None], 0.0)
        hot = torch.zeros_like(z).scatter_(1, at[:, None], 1.0)
        dz = d * (hot - p)
        size = size + p * d.abs()
        lost = lost + d.abs()
        bound = bound + 4 * U * d.abs() * hot
    if dentropy is not None:
        h, H = dentropy.double()[:, None], entropy.double()[:, None]
        dz = dz - torch.where(empty, 0.0, h * p * (fin + H))
        size = size + p * h.abs() * (fin.abs() + H.abs() + 1)
        lost = lost + h.abs() * (88 + H.abs())
    bound = scale * (bound + size * (2 * q + 10 * U) + 2 * 2.0 ** -126 * lost)
    return dz * scale, bound


# ---------------------------------------------------------------- 8-bit activations
def pack(x):
    """The codes and scales of rows, each operation in 32 bits as the format has it, and the values."""
    T, d = x.shape
    v = torch.nn.functional.pad(x.float(), (0, -d % BLOCK)).view(T, -1, BLOCK)
    top = v.abs().amax(2, keepdim=True)
    fine, some = torch.isfinite(top), top >= 1e-30
    # (by a tensor: torch takes a quotient by a number as a product with its reciprocal on the GPU)
    scale = ((top / torch.full_like(top, 127)).view(torch.int32) + 0xFFFF & -0x10000).view(torch.float32)
    scale = torch.where(some, scale, 0.0)
    code = torch.round(torch.where(fine & some, v * (torch.ones_like(scale) / scale), 0.0))
    scale = torch.where(fine, scale, math.nan)
    value = (code * scale).view(T, -1)[:, :d]
    return code.to(torch.int8).view(T, -1)[:, :d], scale[:, :, 0], value


def kept_bound(v, e):
    """How far the kept value of v may be from v when the kernel's own v is off by at most e: half a step of a scale that
    is at most 2^-7 above a 127th of the block's largest, and that largest may be off too.  A code is rounded from a
    product of two roundings: 127 u more."""
    T, d = v.shape
    top = torch.nn.functional.pad(v.abs() + e, (0, -d % BLOCK)).view(T, -1, BLOCK).amax(2, keepdim=True)
    step = top / 127 * (1 + 2.0 ** -7) * (1 + 8 * U)
    most = torch.where(top < 1e-30 * (1 + 8 * U), top, step * (0.5 + 300 * U))  # (a block below 1e-30 is held as zeros)
    return e + most.expand(-1, -1, BLOCK).reshape(T, -1)[:, :d]


__all__ = ["BLOCK", "U", "check", "embed_backward", "embed_forward", "half_step", "kept_bound", "logprob_backward", "logprob_forward",
           "pack"]
