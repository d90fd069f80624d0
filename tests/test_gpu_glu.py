"""twell_glu_forward and _backward against their formulas in 64 bits, element by
element within the bounds of dense_ref.py."""

import pytest

import dense_ref
from helpers import say

pytestmark = pytest.mark.gpu

ACTS = ["relu", "silu", "gelu", "gelu_tanh"]


def _rnd(*shape, dtype, scale=1.0, seed=0):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def _inputs(T, d, F, dtype, seed=0):
    import torch
    dt = getattr(torch, dtype)
    return (_rnd(T, d, dtype=dt, seed=seed), _rnd(F, d, dtype=dt, scale=d ** -0.5, seed=seed + 1),
            _rnd(F, d, dtype=dt, scale=d ** -0.5, seed=seed + 2))


def _nan(*shape, dtype):
    import torch
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def _forward(tw, x, wg, wu, act, save=True):
    T, F = x.shape[0], wg.shape[0]
    h = _nan(T, F, dtype=x.dtype)
    g, u = (_nan(T, F, dtype=x.dtype), _nan(T, F, dtype=x.dtype)) if save else (None, None)
    tw.twell_glu_forward(x, wg, wu, act, h, tw.glu_workspace(T, x.shape[1], F, x.dtype), g=g, u=u)
    return {"h": h, "g": g, "u": u} if save else {"h": h}


def _check_forward(tw, T, d, F, dtype, act, save=True):
    x, wg, wu = _inputs(T, d, F, dtype, seed=T + d + F)
    want = dense_ref.glu_forward(x, wg, wu, act)
    for k, got in _forward(tw, x, wg, wu, act, save).items():
        value, bound = want[k]
        dense_ref.check(got, value, bound + dense_ref.half_step(value.abs() + bound, got.dtype), k)


def _backward(tw, x, wg, wu, g, u, dh, act, dx=True, dw=True):
    T, d = x.shape
    F, dt = wg.shape[0], x.dtype
    ws = tw.glu_backward_workspace(T, d, F, dt)
    ws.fill_(0xFF)  # NaN
    out = {"dx": _nan(T, d, dtype=dt) if dx else None, "dwg": _nan(F, d, dtype=dt) if dw else None,
           "dwu": _nan(F, d, dtype=dt) if dw else None}
    tw.twell_glu_backward(x, wg, wu, g, u, dh, act, out["dx"], out["dwg"], out["dwu"], ws)
    return out


def _check_backward(tw, T, d, F, dtype, act, **parts):
    x, wg, wu = _inputs(T, d, F, dtype, seed=T + d + F)
    g, u, dh = (_rnd(T, F, dtype=x.dtype, scale=s, seed=k) for k, s in ((7, 1.0), (8, 1.0), (9, 0.1)))
    want = dense_ref.glu_backward(x, wg, wu, g, u, dh, act, x.dtype)
    for k, got in _backward(tw, x, wg, wu, g, u, dh, act, **parts).items():
        if got is not None:
            value, bound = want[k]
            dense_ref.check(got, value, bound + dense_ref.half_step(value.abs() + bound, got.dtype), k)


FEW = [1, 2, 15, 16, 17, 31, 33, 48, 50, 63, 64]
SHAPES = ([(t, 128, 192) for t in FEW] + [(1, 64, 64), (3, 2048, 256), (5, 2112, 128), (64, 4160, 64), (65, 64, 64),
          (127, 64, 192), (128, 192, 128), (129, 320, 192), (255, 128, 320), (257, 256, 1024), (1000, 128, 448)])


@pytest.mark.parametrize("shape", SHAPES, ids=["T%d_d%d_F%d" % s for s in SHAPES])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_forward_shapes(gpu_lib, shape, dtype):
    say(f"case glu forward {shape} {dtype}")
    _check_forward(gpu_lib, *shape, dtype, "silu")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T", [7, 300])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_acts(gpu_lib, act, T, dtype):
    say(f"case glu {act} T={T} {dtype}")
    _check_forward(gpu_lib, T, 256, 512, dtype, act, save=False)
    _check_backward(gpu_lib, T, 256, 512, dtype, act)


@pytest.mark.parametrize("T,d,F", [(700, 1024, 2048), (1003, 1024, 4096), (90, 2048, 4096), (600, 64, 8192)])
def test_forward_middle_tiles(gpu_lib, T, d, F):
    say(f"case glu forward middle tiles T={T} d={d} F={F}")
    _check_forward(gpu_lib, T, d, F, "bfloat16", "silu")


@pytest.mark.parametrize("shape", [(128, 4096, 512), (70, 2112, 64), (100, 4096, 1024), (513, 2048, 320)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_forward_split(gpu_lib, shape, dtype):
    """Few tiles and a long d: K is split and the parts joined in a workspace, without which the call is refused."""
    import torch
    say(f"case glu forward split {shape} {dtype}")
    T, d, F = shape
    assert gpu_lib.twell_glu_workspace_bytes(T, d, F, getattr(torch, dtype)) > 0
    _check_forward(gpu_lib, *shape, dtype, "gelu")
    _check_forward(gpu_lib, *shape, dtype, "relu", save=False)
    x, wg, wu = _inputs(T, d, F, dtype)
    with pytest.raises(gpu_lib.TwellError):
        gpu_lib.twell_glu_forward(x, wg, wu, "relu", torch.empty((T, F), dtype=x.dtype, device="cuda"))


@pytest.mark.parametrize("T,F", [(8192, 1024), (4097, 1600), (2049, 3008)])
def test_forward_large_tiles(gpu_lib, T, F):
    say(f"case glu forward large tiles T={T} F={F}")
    _check_forward(gpu_lib, T, 512, F, "bfloat16", "gelu")


BACKWARD = [(1, 64, 64), (2, 128, 64), (63, 64, 128), (64, 192, 64), (65, 64, 192), (130, 320, 448), (500, 128, 2048),
            (1003, 1024, 512), (16, 2048, 4096), (2000, 64, 64)]


@pytest.mark.parametrize("shape", BACKWARD, ids=["T%d_d%d_F%d" % s for s in BACKWARD])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_backward_shapes(gpu_lib, shape, dtype):
    say(f"case glu backward {shape} {dtype}")
    _check_backward(gpu_lib, *shape, dtype, "silu")


@pytest.mark.parametrize("shape", [(1003, 1024, 4096), (4096, 1024, 1024), (300, 4096, 2048), (4000, 4096, 256), (200, 2112, 6400),
                                    (12300, 1024, 128), (4097, 3008, 64)])
def test_backward_large_tiles(gpu_lib, shape):
    say(f"case glu backward large tiles {shape}")
    _check_backward(gpu_lib, *shape, "bfloat16", "gelu_tanh")


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_backward_parts(gpu_lib, dtype):
    say("case glu backward parts")
    _check_backward(gpu_lib, 100, 128, 192, dtype, "silu", dw=False)
    _check_backward(gpu_lib, 100, 128, 192, dtype, "silu", dx=False)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_no_rows(gpu_lib, dtype):
    """T = 0: h has no rows, the weights' gradients are 0."""
    import torch
    say("case glu T=0")
    x, wg, wu = _inputs(0, 128, 192, dtype)
    _forward(gpu_lib, x, wg, wu, "silu")
    e = torch.empty((0, 192), dtype=x.dtype, device="cuda")
    got = _backward(gpu_lib, x, wg, wu, e, e, e, "silu")
    assert not got["dwg"].any() and not got["dwu"].any()


@pytest.mark.parametrize("act", ACTS)
def test_far_values(gpu_lib, act):
    """g far outside the exponentials' range: act(g) is 0 or g, its slope 0 or 1."""
    import torch
    say(f"case glu far values {act}")
    d = 64
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.zeros((8, d), dtype=dtype, device="cuda")
        x[:, 0] = torch.tensor([-1e30, -3e4, -200.0, -0.0, 0.0, 200.0, 3e4, 1e30], device="cuda")
        w = torch.zeros((64, d), dtype=dtype, device="cuda")
        w[:, 0] = 1.0
        wu = torch.zeros_like(w)
        x[:, 1], wu[:, 1] = 1.0, 2.0  # u = 2
        got = _forward(gpu_lib, x, w, wu, act)
        g = got["g"][:, 0].float()
        assert torch.equal(got["h"][:, 0].float(), torch.where(g > 100, 2 * g, torch.zeros_like(g)))
        one = torch.ones_like(got["g"])
        grad = _backward(gpu_lib, x, w, wu, got["g"], got["u"], one, act)
        assert torch.isfinite(grad["dx"]).all()
        # dx[:, 0] = sum over the 64 neurons of dh u act'(g)
        slope = grad["dx"][:, 0].float() / 128
        half = 0.0 if act == "relu" else 0.5
        want = torch.tensor([0, 0, 0, half, half, 1, 1, 1], device="cuda", dtype=torch.float32)
        assert torch.equal(slope, want), slope


def test_non_finite_row_stays_alone(gpu_lib):
    import torch
    say("case glu non-finite row")
    for T in (5, 40, 300):
        x, wg, wu = _inputs(T, 128, 192, "bfloat16")
        good = _forward(gpu_lib, x, wg, wu, "silu")["h"]
        x[3, 5] = float("nan")
        wg[7, 1] = float("inf")
        bad = _forward(gpu_lib, x, wg, wu, "silu")["h"]
        rows, cols = [i for i in range(T) if i != 3], [i for i in range(192) if i != 7]
        assert torch.equal(bad[rows][:, cols], good[rows][:, cols])
        assert torch.isnan(bad[3]).all()


@pytest.mark.parametrize("T,d,F", [(1, 64, 64), (65, 64, 192), (1003, 1024, 512), (2000, 512, 2048)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_infinite_last_row(gpu_lib, T, d, F, dtype):
    """An infinity in x's last row gives infinite gradients of the weights, and no NaN from rows that are not there."""
    import torch
    say(f"case glu infinite last row {T} {d} {F} {dtype}")
    x, wg, wu = _inputs(T, d, F, dtype)
    x[-1, 3] = float("inf")
    one = torch.ones((T, F), dtype=x.dtype, device="cuda")
    got = _backward(gpu_lib, x, wg, wu, one, one, one, "relu", dx=False)
    for k in ("dwg", "dwu"):
        assert (got[k][:, 3] == float("inf")).all() and torch.isfinite(got[k][:, :3]).all() and torch.isfinite(got[k][:, 4:]).all(), k


def test_same_bits_on_a_stream(gpu_lib):
    import torch
    say("case glu same bits")
    x, wg, wu = _inputs(700, 1024, 2048, "bfloat16")
    dh = _rnd(700, 2048, dtype=x.dtype, seed=5)
    first = _forward(gpu_lib, x, wg, wu, "silu")
    grads = _backward(gpu_lib, x, wg, wu, first["g"], first["u"], dh, "silu")
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        again = _forward(gpu_lib, x, wg, wu, "silu")
        grads2 = _backward(gpu_lib, x, wg, wu, first["g"], first["u"], dh, "silu")
        torch.cuda.current_stream().synchronize()
    for a, b in ((first, again), (grads, grads2)):
        for k in a:
            assert torch.equal(a[k], b[k]), k


def test_past_32_bits(gpu_lib):
    """Results and stored products whose offsets do not fit 32 bits."""
    import torch
    T, d, F = (1 << 32) // 32768 + 260, 64, 32768
    say(f"case glu T={T} F={F}")
    x = torch.zeros((T, d), dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1.0
    x[-1, 0] = 2.0
    w = torch.zeros((F, d), dtype=torch.bfloat16, device="cuda")
    w[:, 0] = 1.0
    w[-1, 0] = 3.0
    h = torch.zeros((T, F), dtype=torch.bfloat16, device="cuda")
    gpu_lib.twell_glu_forward(x, w, w, "relu", h)
    assert (h[-2, :-1] == 1).all() and (h[-1, :-1] == 4).all() and h[-1, -1] == 36 and (h[0, :-1] == 1).all()
    dx = torch.zeros_like(x)
    dw, dwu = torch.zeros_like(w), torch.zeros_like(w)
    g = h  # any stored product: here g = u = h
    dh = torch.ones_like(h[:1]).expand(T, F).contiguous()
    ws = gpu_lib.glu_backward_workspace(T, d, F, torch.bfloat16)
    gpu_lib.twell_glu_backward(x, w, w, g, g, dh, "relu", dx, dw, dwu, ws)
    # dg = u = h, du = h: dx[t][0] = 2 sum_j h[t][j] w[j][0], dw[j][0] = sum_t h[t][j] x[t][0]
    want = 2 * ((F - 1) * 4.0 + 36 * 3)
    assert abs(dx[-1, 0].item() - want) <= want * 2.0 ** -8
    want = (T - 1) * 1.0 + 4 * 2
    assert abs(dw[0, 0].item() - want) <= want * 2.0 ** -8 and abs(dwu[F - 2, 0].item() - want) <= want * 2.0 ** -8


def test_refusals(gpu_lib):
    import torch
    tw = gpu_lib
    x, wg, wu = _inputs(4, 64, 128, "bfloat16")
    h = torch.empty((4, 128), dtype=torch.bfloat16, device="cuda")
    for args, kw, err in (((x, wg, wu[:64], "silu", h), {}, ValueError), ((x, wg, wu, "swish", h), {}, ValueError),
                          ((x, wg, wu, "silu", h.float()), {}, TypeError), ((x, wg.float(), wu, "silu", h), {}, TypeError),
                          ((x, wg, wu, "silu", h.t()), {}, ValueError), ((x, wg, wu, "silu", h.cpu()), {}, ValueError),
                          ((x, wg, wu, "silu", h), {"g": h[:2]}, ValueError),
                          ((x.half(), wg.half(), wu.half(), "silu", h.half()), {}, TypeError)):
        with pytest.raises(err):
            tw.twell_glu_forward(*args, **kw)
    odd = [t[:, :32].contiguous() for t in (x, wg, wu)]
    with pytest.raises(tw.TwellError):
        tw.twell_glu_forward(*odd, "silu", h)
    flat = torch.empty(4 * 128 + 1, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(tw.TwellError):
        tw.twell_glu_forward(x, wg, wu, "silu", flat[1:].view(4, 128))
    with pytest.raises(tw.TwellError):  # dwg without dwu
        tw.twell_glu_backward(x, wg, wu, h, h, h, "silu", None, wg.clone(), None, tw.glu_backward_workspace(4, 64, 128, x.dtype))
    with pytest.raises(tw.TwellError):  # no workspace
        tw.twell_glu_backward(x, wg, wu, h, h, h, "silu", x.clone(), None, None, None)
    for ws in (torch.empty(1 << 20, dtype=torch.uint8), torch.empty((1 << 11, 1 << 10), dtype=torch.uint8, device="cuda").t()):
        with pytest.raises(ValueError):
            tw.twell_glu_backward(x, wg, wu, h, h, h, "silu", x.clone(), None, None, ws)
