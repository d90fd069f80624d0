"""Log probabilities of confident rows: one logit far above the others, so that L = log sum exp(c (z - m)) is small.  L, the
entropy and 1 - p of that token are right relative to themselves, by every kernel that takes a row."""

import math

import pytest

import tokens_ref
from helpers import say
from tokens_ref import U

pytestmark = pytest.mark.gpu

# a wave's row (short, longer), a workgroup's in one round, cut into segments, and in several rounds
ROWS = [(3, 1), (3, 64), (5, 1027), (5, 2048), (2050, 4001), (3, 8000), (3, 12289), (2, 30001), (1, 131072), (1100, 26003)]


def _logits(T, V, dtype, more, scale, seed=0):
    """Rows whose S - 1 is about `more`: one logit of 3 (or of two equal ones in every fifth row), at a place of the row's own,
    over others within 1 of each other."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed + V)
    gap = math.log(max(V - 1, 1) / more) / scale
    z = 3 - gap + torch.rand((T, V), generator=gen, device="cuda") - 0.5
    at = torch.randint(0, V, (T,), generator=gen, device="cuda")
    at[0], at[-1] = V - 1, 0
    z[torch.arange(T, device="cuda"), at] = 3
    z[4::5, V // 3] = 3
    return z.to(getattr(torch, dtype)), at


def _want(z, scale):
    """{name: (value, bound)} in 64 bits.  The terms of s = S - n and of W are of one sign, each with the error of its
    exponential (3 + 4 |x| roundings) and at most V / 256 + 74 additions and V / 1024 + 74 scalings by a larger maximum after
    it: tokens_ref.logprob_forward's count K holds for s itself.  log(1 + y) and the sums of n - 1 and 1 are 8 u more."""
    import torch
    x = (z.double() - z.double().amax(1, keepdim=True)) * scale
    top = x == 0
    s = torch.where(top, 0.0, torch.exp(x)).sum(1)
    W = (torch.exp(x) * -x).sum(1)
    more = s + top.sum(1) - 1
    L, mean = torch.log1p(more), W / (1 + more)
    K = z.shape[1] / 128 + 8 * (-x / math.log(2)).amax(1).clamp_max(200) + 450
    return {"L": (L, L * (K + 8) * U), "entropy": (L + mean, L * (K + 8) * U + mean * (2 * K + 30) * U + 2 * U * (L + mean)),
            "logp": (-L, L * (K + 8) * U)}


def _forward(tw, z, targets, scale, k=0):
    import torch
    T, V = z.shape
    new = lambda *s: torch.full(s, 7.25, device="cuda")  # noqa: E731
    norm, entropy, logp, top = new(T, 2), new(T), new(T), new(T, k) if k else None
    idx = torch.empty((T, k), dtype=torch.int32, device="cuda") if k else None
    tw.twell_logprob_forward(z, targets, logp, norm, tw.logprob_workspace(T, V, k), scale=scale, entropy=entropy, top_logp=top,
                             top_idx=idx)
    return {"norm": norm, "L": norm[:, 1].contiguous(), "entropy": entropy, "logp": logp, "top": top}


@pytest.mark.parametrize("more", [1e-7, 1e-6, 3e-5, 1e-3, 0.3])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_forward(gpu_lib, dtype, more):
    import torch
    for T, V in ROWS:
        for scale in (1.0, 0.7):
            say(f"case logprob confident T={T} V={V} {dtype} {more} {scale}")
            z, at = _logits(T, V, dtype, more, scale)
            want = _want(z, float(torch.tensor(scale, dtype=torch.float32)))
            for k in sorted({0, min(V, 3)}):
                got = _forward(gpu_lib, z, at, scale, k)
                for name, (value, bound) in want.items():
                    tokens_ref.check(got[name], value, bound, name)
                if k:
                    tokens_ref.check(got["top"][:, 0].contiguous(), *want["logp"], "top_logp")
            value, bound = want["L"]
            assert (bound <= 0.01 * value).all()  # (an L of 0 fails)


@pytest.mark.parametrize("more", [1e-7, 1e-6, 3e-5, 1e-3, 0.3])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_gradient_of_the_likely_token(gpu_lib, dtype, more):
    """dz of the target that is the largest: c dlogp (1 - p), p = exp(-L) from the stored L.  L log2(e), back to the natural
    logarithm, expm1 and the products with c and dlogp are at most 14 u of it.  The row's other gradients are as any row's."""
    import torch
    for T, V in ROWS:
        for scale in (1.0, 0.7):
            say(f"case logprob confident gradient T={T} V={V} {dtype} {more} {scale}")
            z, at = _logits(T, V, dtype, more, scale)
            got = _forward(gpu_lib, z, at, scale)
            gen = torch.Generator(device="cuda").manual_seed(1)
            dlogp, dent = (torch.randn(T, generator=gen, device="cuda") for _ in range(2))
            dz = torch.full_like(z, math.nan)
            gpu_lib.twell_logprob_backward(z, at, got["norm"], dlogp, dz, scale=scale)
            c = float(torch.tensor(scale, dtype=torch.float32))
            value = c * dlogp.double() * -torch.expm1(-got["L"].double())
            tokens_ref.check(dz.gather(1, at[:, None])[:, 0], value, 14 * U * value.abs(), "dz of the target")
            for parts in ((dlogp, None), (dlogp, dent)):
                want, bound = tokens_ref.logprob_backward(z, at, got["norm"], parts[0], c, got["entropy"], parts[1])
                gpu_lib.twell_logprob_backward(z, at, got["norm"], parts[0], dz, scale=scale, entropy=got["entropy"],
                                               dentropy=parts[1])
                tokens_ref.check(dz, want, bound, "dlogits")
