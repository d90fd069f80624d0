"""The dense operators' workspaces: one for the most rows serves every call with fewer."""

import ctypes

import pytest

import unstructured_sparse_transformer_amd as tw
from helpers import say

AT = 4096  # an aligned, never dereferenced fake device address
ALIGN, WORKSPACE = -2, -6
# row counts around the tiles' and the row groups' edges, and a spread of others
ROWS = sorted({m + i for m in [64 * k for k in range(1, 41)] + [1 << k for k in range(12, 15)] for i in (-1, 0, 1)}
              | set(range(1, 300)) | set(range(301, 20000, 97)))
GLU = [(64, 64), (128, 448), (384, 1536), (512, 512), (1024, 4096), (2048, 2048), (2048, 8192), (4096, 256), (64, 8192)]
NORM = [1, 16, 17, 64, 200, 256, 512, 513, 1001, 1024, 2048, 4096, 8191, 8192]


def _grows(size):
    last = 0
    for T in ROWS:
        n = size(T)
        assert n >= last, f"T={T}: {n} bytes, {last} for fewer rows"
        last = n


@pytest.mark.parametrize("d,F", GLU)
@pytest.mark.parametrize("vd", [0, 1])
def test_gated_product_sizes_grow(d, F, vd):
    lib = tw.load()
    for size in (lib.twell_glu_workspace_bytes, lib.twell_glu_backward_workspace_bytes):
        _grows(lambda T: size(T, d, F, vd))


@pytest.mark.parametrize("d", NORM)
def test_block_norm_sizes_grow(d):
    _grows(lambda T: tw.load().twell_block_norm_workspace_bytes(T, d))


@pytest.mark.parametrize("most", [300, 1003, 8192, 20000])
def test_gated_product_takes_the_largest(most):
    """A workspace that is large enough but starts 16 bytes too late is refused for its alignment, one byte less than
    a call's own rows need for its size."""
    lib = tw.load()
    for d, F in GLU:
        for vd in (0, 1):
            n = lib.twell_glu_backward_workspace_bytes(most, d, F, vd)
            call = lambda T, n: lib.twell_glu_backward(*[AT] * 6, T, d, F, vd, 1, AT, AT, AT, AT + 16, n, None)  # noqa: E731
            for T in ROWS:
                assert T > most or call(T, n) == ALIGN, (T, d, F, vd)
            assert call(most, 1024) == WORKSPACE


@pytest.mark.parametrize("most", [64, 777, 6141, 8192, 20000])
def test_block_norm_takes_the_largest(most):
    lib = tw.load()
    for d in NORM:
        n = lib.twell_block_norm_workspace_bytes(most, d)

        def call(T, n):
            bn = tw.TwellBlockNormT(T=T, d=d, eps=1e-6, alpha=1.0)
            return lib.twell_block_norm_backward(ctypes.byref(bn), AT, None, AT, AT, 0, AT, None, None, *[None] * 4,
                                                 AT + 16, n, None)
        for T in ROWS:
            assert T > most or call(T, n) == ALIGN, (T, d)
        assert call(most, 16) == WORKSPACE


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_one_workspace_for_every_batch(gpu_lib, dtype):
    """The same bits as with a workspace of the batch's own, batches that split their products' K among them."""
    import torch
    dt, d, F, most = getattr(torch, dtype), 2048, 512, 1500
    gen = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dt)  # noqa: E731
    x, wg, wu, dh = rnd(most, d), rnd(F, d) * d ** -0.5, rnd(F, d) * d ** -0.5, rnd(most, F)
    one = (tw.glu_workspace(most, d, F, dt), tw.glu_backward_workspace(most, d, F, dt), tw.block_norm_workspace(most, d))

    def step(T, ws):
        h, g, u = (torch.empty((T, F), dtype=dt, device="cuda") for _ in range(3))
        tw.twell_glu_forward(x[:T], wg, wu, "silu", h, ws[0], g=g, u=u)
        dx, dres, dwg, dwu = (torch.empty_like(t) for t in (x[:T], x[:T], wg, wu))
        tw.twell_glu_backward(x[:T], wg, wu, g, u, dh[:T], "silu", dx, dwg, dwu, ws[1])
        dw = torch.empty(d, device="cuda")
        tw.twell_block_norm_backward(tw.BlockNorm(), x[:T], None, None, dx, dres, None, ws[2], dw_pre=dw)
        return h, g, u, dx, dwg, dwu, dres, dw

    for T in (1, 64, 65, 130, 257, 700, 1499, 1500):
        say(f"case one workspace {dtype} T={T}")
        own = (tw.glu_workspace(T, d, F, dt), tw.glu_backward_workspace(T, d, F, dt), tw.block_norm_workspace(T, d))
        for a, b in zip(step(T, own), step(T, one)):
            assert torch.equal(a, b)
