"""How the gated product that keeps g and u in 8 bits is cut up: K is split as twell_glu_forward splits it from 65 rows
on, so that h has the same bits."""

import math
import random

import pytest

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
