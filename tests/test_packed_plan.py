"""How the gated product that keeps g and u in 8 bits is cut up: K is split as twell_glu_forward splits it from 65 rows
on, so that h has the same bits, and every tile keeps the codes with and without the sign."""

import math
import random

import pytest

import dense_ref
import tokens_ref
import unstructured_sparse_transformer_amd as tw
from helpers import say

# the first ones: sizes where the least estimated time alone would split K differently
SIZES = [(129, 3328, 6528), (1249, 4032, 896), (129, 3904, 7936), (293, 3712, 3584), (8545, 3968, 128), (65, 64, 64),
         (100, 128, 192), (128, 4096, 512), (700, 1024, 2048), (1003, 1024, 4096), (70, 2112, 64)]


def test_workspaces_show_the_same_splits():
    """A workspace of up to T rows is the splits' parts at most, of calls up to 64 rows (whose twell_glu_forward needs
    none) and of calls beyond, where the two calls have the same splits."""
    lib, rng = tw.load(), random.Random(5)
    more = [(rng.randint(65, 9000), 64 * rng.randint(1, 64), 64 * rng.randint(1, 128)) for _ in range(1000)]
    for T, d, F in SIZES + more:
        plain, packed = (lambda t: lib.twell_glu_workspace_bytes(t, d, F, tw.TWELL_BF16)), lambda t: lib.twell_glu_packed_workspace_bytes(t, d, F)
        assert plain(64) == 0
        assert packed(T) == max(packed(64), plain(T)), (T, d, F)


@pytest.mark.gpu
@pytest.mark.parametrize("T,d,F", SIZES, ids=["T%d_d%d_F%d" % s for s in SIZES])
def test_h_has_the_bits_of_the_gated_product(gpu_lib, T, d, F):
    import torch
    say(f"case packed plan h T={T} d={d} F={F}")
    gen = torch.Generator(device="cuda").manual_seed(T)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    x, wg, wu = rnd(T, d), rnd(F, d) * d ** -0.5, rnd(F, d) * d ** -0.5
    want, got = (torch.full((T, F), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    tw.twell_glu_forward(x, wg, wu, "silu", want, tw.glu_workspace(T, d, F, x.dtype))
    g, u = tw.PackedAct.empty(T, F), tw.PackedAct.empty(T, F)
    tw.twell_glu_forward_packed(x, wg, wu, "silu", got, g, u, tw.glu_packed_workspace(T, d, F))
    assert torch.isfinite(want).all() and torch.equal(got, want)


# by workgroups' tile: 256 x 256, 256 x 128, 128 x 128 (three), 128 x 64 (two), and K in 8 parts
TILES = [(8192, 256, 1024), (1003, 1024, 4096), (700, 1024, 2048), (65, 64, 64), (1249, 4032, 896), (100, 128, 192), (33, 256, 512), (128, 4096, 512)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,d,F", TILES, ids=["T%d_d%d_F%d" % s for s in TILES])
def test_codes_of_every_tile(gpu_lib, T, d, F):
    """ReLU's codes against the product in 64 bits: within half a step and the product's own error (tokens_ref), with
    keep_sign a g above 0 whose code is 0 has 1, and all else is as without.  A g nearer to 0 than the product's error may
    have either sign."""
    import torch
    say(f"case packed plan codes T={T} d={d} F={F}")
    gen = torch.Generator(device="cuda").manual_seed(d)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    x, wg, wu = rnd(T, d), rnd(F, d) * d ** -0.5, rnd(F, d) * d ** -0.5
    got = {}
    for keep in (False, True):
        h, g, u = torch.full((T, F), math.nan, dtype=torch.bfloat16, device="cuda"), tw.PackedAct.empty(T, F), tw.PackedAct.empty(T, F)
        for p in (g, u):
            p.code.fill_(-77)
            p.scale.fill_(math.nan)
        tw.twell_glu_forward_packed(x, wg, wu, "relu", h, g, u, tw.glu_packed_workspace(T, d, F), keep_sign=keep)
        got[keep] = h, g, u
    (h, g, u), (h1, g1, u1) = got[False], got[True]
    want = dense_ref.glu_forward(x, wg, wu, "relu")
    tokens_ref.check(h, *want["h"], "h")
    for name, p in (("g", g), ("u", u)):
        value = p.code.double() * p.scale.double().repeat_interleave(32, 1)
        assert ((value - want[name][0]).abs() <= tokens_ref.kept_bound(*want[name])).all(), name
    assert torch.equal(h, h1) and torch.equal(u.code, u1.code) and torch.equal(u.scale, u1.scale) and torch.equal(g.scale, g1.scale)
    exact, bound = want["g"]
    sure = exact.abs() > bound
    raised = (g.code == 0) & (exact > 0)
    assert raised.any() and torch.equal(g1.code[sure], torch.where(raised, torch.ones_like(g.code), g.code)[sure])
    # (the bound of the product, d 2^-24 of its terms' magnitudes or more, reaches half a step at d = 4032: codes of -1 and
    # 1 are among those of unsure sign, and keep_sign changes zeros only)
    assert torch.equal(g1.code[g.code != 0], g.code[g.code != 0])
    assert ((g1.code[g.code == 0] == 0) | (g1.code[g.code == 0] == 1)).all()
