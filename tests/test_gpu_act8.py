"""Activations kept in 8 bits: packing bit by bit against the format, and the gated
product that keeps g and u so against its formulas in 64 bits."""

import math

import pytest

import dense_ref
import tokens_ref
from helpers import say

pytestmark = pytest.mark.gpu

TYPES = ["bfloat16", "float32"]
ACTS = ["relu", "silu", "gelu", "gelu_tanh"]


def _rnd(*shape, dtype="bfloat16", scale=1.0, seed=0):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(getattr(torch, dtype))


def _packed(tw, T, d):
    """A PackedAct of 0xFF bytes, between others that have to stay."""
    import torch
    nb = -(-d // 32)
    code = torch.full((T * d + 128,), -1, dtype=torch.int8, device="cuda")
    scale = torch.full((T * nb + 128,), math.nan, dtype=torch.bfloat16, device="cuda")
    return tw.PackedAct(code[64:64 + T * d].view(T, d), scale[64:64 + T * nb].view(T, nb)), code, scale


def _check_pack(tw, x):
    import torch
    T, d = x.shape
    p, code, scale = _packed(tw, T, d)
    tw.twell_act_pack(x, p)
    want_code, want_scale, want = tokens_ref.pack(x)
    fine = torch.isfinite(want)
    assert torch.equal(p.code[fine], want_code[fine])
    assert torch.equal(p.scale.float().nan_to_num(-1), want_scale.nan_to_num(-1))
    assert (code[:64] == -1).all() and (code[64 + T * d:] == -1).all()
    assert torch.isnan(scale[:64]).all() and torch.isnan(scale[64 + p.scale.numel():]).all()
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.full((T, d), 7.25, dtype=dtype, device="cuda")
        tw.twell_act_unpack(p, out)
        assert torch.equal(out.float().nan_to_num(-77), want.to(dtype).float().nan_to_num(-77))
    off = (want.double() - x.double()).abs()
    assert (off <= tokens_ref.kept_bound(x.double().nan_to_num(0, 0, 0), 0.0))[fine].all()


SHAPES = [(1, 1), (1, 31), (2, 32), (3, 33), (5, 3), (7, 64), (64, 1001), (9, 65), (300, 96), (1000, 8), (33, 4096), (1, 20000), (4097, 36)]


@pytest.mark.parametrize("shape", SHAPES, ids=["T%d_d%d" % s for s in SHAPES])
@pytest.mark.parametrize("dtype", TYPES)
def test_pack(gpu_lib, shape, dtype):
    say(f"case act pack {shape} {dtype}")
    _check_pack(gpu_lib, _rnd(*shape, dtype=dtype, seed=shape[1]))


@pytest.mark.parametrize("dtype", TYPES)
def test_pack_values(gpu_lib, dtype):
    """Zeros, -0, single large values, values of every size, halves between codes, the type's largest, NaN, infinities."""
    import torch
    say(f"case act pack values {dtype}")
    x = _rnd(40, 160, dtype=dtype)
    x[0] = 0
    x[1] = -0.0
    x[2, 5] = 1e4
    x[3] *= 1e30
    x[4] *= 1e-25
    x[5] *= 1e-31
    x[6] *= 1e-38
    x[7, :32] = torch.arange(32, device="cuda") + 0.5
    x[7, 0] = 127
    x[8, 3] = torch.finfo(x.dtype).max
    x[9, 40] = math.nan
    x[10, 0] = math.inf
    x[11, 159] = -math.inf
    x[12] = math.nan
    x[13] = torch.finfo(x.dtype).tiny
    x[14:] *= torch.exp2(torch.arange(26, device="cuda") * 4 - 52)[:, None].to(x.dtype)
    _check_pack(gpu_lib, x)


def test_pack_past_32_bits(gpu_lib):
    import torch
    T, d = 70000, 32768
    say("case act pack, 2.3e9 elements")
    x = torch.zeros((T, d), dtype=torch.bfloat16, device="cuda")
    x[-1] = _rnd(1, d)[0]
    p = gpu_lib.PackedAct.empty(T, d)
    gpu_lib.twell_act_pack(x, p)
    code, scale, want = tokens_ref.pack(x[-1:])
    assert torch.equal(p.code[-1:], code) and torch.equal(p.scale[-1:].float(), scale)
    x.fill_(1)
    gpu_lib.twell_act_unpack(p, x)
    assert torch.equal(x[-1:], want.bfloat16()) and not x[:-1].any()


# ---------------------------------------------------------------- the gated product
def _inputs(T, d, F):
    s = T + d + F
    return (_rnd(T, d, seed=s), _rnd(F, d, scale=d ** -0.5, seed=s + 1), _rnd(F, d, scale=d ** -0.5, seed=s + 2))


def _nan(*shape):
    import torch
    return torch.full(shape, math.nan, dtype=torch.bfloat16, device="cuda")


def _value(p):
    """What a PackedAct stands for."""
    T, d = p.code.shape
    return p.code.double() * p.scale.double().repeat_interleave(32, 1)[:, :d]


def _forward(tw, x, wg, wu, act, most=None):
    T, d = x.shape
    F = wg.shape[0]
    h, (g, *g_around), (u, *u_around) = _nan(T, F), _packed(tw, T, F), _packed(tw, T, F)
    ws = tw.glu_packed_workspace(most or T, d, F)
    if ws is not None:
        ws.fill_(0xFF)
    tw.twell_glu_forward_packed(x, wg, wu, act, h, g, u, ws)
    for code, scale in (g_around, u_around):
        assert (code[:64] == -1).all() and (code[64 + T * F:] == -1).all() and scale[:64].isnan().all()
        assert scale[64 + g.scale.numel():].isnan().all()
    return h, g, u


def _check(tw, T, d, F, act, backward=True):
    import torch
    x, wg, wu = _inputs(T, d, F)
    h, g, u = _forward(tw, x, wg, wu, act)
    want = dense_ref.glu_forward(x, wg, wu, act)
    value, bound = want["h"]
    tokens_ref.check(h, value, bound, "h")
    for name, p in (("g", g), ("u", u)):
        v, e = want[name]
        off = (_value(p) - v).abs()
        most = tokens_ref.kept_bound(v, e)
        assert (off <= most).all(), f"{name}: off by {float((off / most).max()):.3g} bounds"
        assert torch.equal(p.code.abs().view(T, -1, 32).amax(2) >= 126, p.scale > 0)  # the largest of a block fills its scale
    if not backward:
        return
    dh = _rnd(T, F, scale=0.1, seed=9)
    dx, dwg, dwu, again = _nan(T, d), _nan(F, d), _nan(F, d), _nan(T, F)
    ws = tw.glu_backward_workspace(T, d, F, torch.bfloat16)
    ws.fill_(0xFF)
    tw.twell_glu_backward_packed(x, wg, wu, g, u, dh, act, dx, dwg, dwu, ws, h=again)
    gv, uv = _value(g), _value(u)
    want = dense_ref.glu_backward(x, wg, wu, gv, uv, dh, act, torch.bfloat16)
    a = dense_ref.act(gv, act)
    want["h"] = a * uv, 4e-6 * (1 + gv.abs()) * uv.abs()
    for name, got in (("dx", dx), ("dwg", dwg), ("dwu", dwu), ("h", again)):
        value, bound = want[name]
        tokens_ref.check(got, value, bound, name)


GLU = [(1, 64, 64), (2, 128, 192), (31, 64, 128), (64, 192, 64), (65, 64, 64), (127, 64, 192), (129, 320, 192), (257, 256, 1024),
       (1000, 128, 448), (128, 4096, 512), (70, 2112, 64), (513, 2048, 320), (700, 1024, 2048), (1003, 1024, 4096), (2049, 512, 3008)]


@pytest.mark.parametrize("shape", GLU, ids=["T%d_d%d_F%d" % s for s in GLU])
def test_glu_packed(gpu_lib, shape):
    say(f"case glu packed {shape}")
    _check(gpu_lib, *shape, "silu")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T", [7, 300])
def test_glu_packed_acts(gpu_lib, act, T):
    say(f"case glu packed {act} T={T}")
    _check(gpu_lib, T, 256, 512, act)


@pytest.mark.parametrize("T,F", [(4097, 1600), (8192, 1024)])
def test_glu_packed_large_tiles(gpu_lib, T, F):
    say(f"case glu packed large tiles T={T} F={F}")
    _check(gpu_lib, T, 512, F, "gelu", backward=False)


@pytest.mark.parametrize("T,d,F", [(100, 128, 256), (1003, 1024, 4096), (5000, 256, 2048)])
def test_h_is_the_gated_product_s(gpu_lib, T, d, F):
    """h has the bits of twell_glu_forward's (from 65 rows on, where both run the same product)."""
    import torch
    say(f"case glu packed h T={T} d={d} F={F}")
    x, wg, wu = _inputs(T, d, F)
    h = _nan(T, F)
    gpu_lib.twell_glu_forward(x, wg, wu, "gelu", h, gpu_lib.glu_workspace(T, d, F, x.dtype))
    assert torch.equal(_forward(gpu_lib, x, wg, wu, "gelu")[0], h)


@pytest.mark.parametrize("T,d,F", [(100, 128, 192), (300, 256, 512), (128, 4096, 512), (1003, 1024, 4096), (8192, 512, 1024)])
def test_glu_packed_keeps_the_sign(gpu_lib, T, d, F):
    """keep_sign: the codes of g that are 0 for a g above 0 are 1, all others, u and h as without; and ReLU's gradients
    are as far from those of the exact g and u as the others' roundings: half a step is 2^-8 of a block's largest, about
    2^-6.5 of its typical value, and bf16's 2^-8 enter twice: 2% of the 2-norm are allowed."""
    import torch
    say(f"case glu packed keep_sign {T} {d} {F}")
    x, wg, wu = _inputs(T, d, F)
    plain = _forward(gpu_lib, x, wg, wu, "relu")
    h, (g, *_), (u, *_) = _nan(T, F), _packed(gpu_lib, T, F), _packed(gpu_lib, T, F)
    gpu_lib.twell_glu_forward_packed(x, wg, wu, "relu", h, g, u, gpu_lib.glu_packed_workspace(T, d, F), keep_sign=True)
    for a, b in ((h, plain[0]), (u.code, plain[2].code), (u.scale, plain[2].scale), (g.scale, plain[1].scale)):
        assert torch.equal(a, b)
    exact, bound = dense_ref.glu_forward(x, wg, wu, "relu")["g"]
    sure = exact.abs() > bound
    raised = (plain[1].code == 0) & (exact > 0)
    want = torch.where(raised, torch.ones_like(g.code), plain[1].code)
    assert torch.equal(g.code[sure], want[sure]) and raised.any()
    dh = _rnd(T, F, seed=3)
    got = _nan(T, d), _nan(F, d), _nan(F, d)
    gpu_lib.twell_glu_backward_packed(x, wg, wu, g, u, dh, "relu", *got, gpu_lib.glu_backward_workspace(T, d, F, torch.bfloat16))
    uv, xd = x.double() @ wu.double().T, x.double()
    dg, du = dh.double() * uv * (exact > 0), dh.double() * exact.clamp_min(0)
    for a, b in zip(got, (dg @ wg.double() + du @ wu.double(), dg.T @ xd, du.T @ xd)):
        assert float((a.double() - b).norm() / b.norm()) < 0.02


def test_glu_packed_bad_rows(gpu_lib):
    """NaN and infinities in x spoil the kept values of their own rows only."""
    import torch
    say("case glu packed bad rows")
    for T, d, F in ((200, 128, 192), (100, 4096, 512)):  # whole, and K split
        x, wg, wu = _inputs(T, d, F)
        clean = _forward(gpu_lib, x, wg, wu, "silu")
        x[3, 5], x[T - 1, 0] = math.nan, math.inf
        got = _forward(gpu_lib, x, wg, wu, "silu")
        rows = torch.ones(T, dtype=torch.bool, device="cuda")
        rows[3] = rows[T - 1] = False
        for a, b in zip(got[1:], clean[1:]):
            assert torch.isnan(_value(a)[~rows]).all()
            assert torch.equal(a.code[rows], b.code[rows]) and torch.equal(a.scale[rows], b.scale[rows])


def test_glu_packed_parts(gpu_lib):
    """Each gradient by itself, and h by itself, has the bits that it has with the others; a step in a captured graph too."""
    import torch
    tw = gpu_lib
    say("case glu packed parts")
    T, d, F = 333, 256, 512
    x, wg, wu = _inputs(T, d, F)
    h, g, u = _forward(tw, x, wg, wu, "silu")
    dh, ws = _rnd(T, F, seed=4), tw.glu_backward_workspace(2 * T, d, F, torch.bfloat16)
    back = lambda dx=None, dw=(None, None), h=None: tw.twell_glu_backward_packed(x, wg, wu, g, u, dh, "silu", dx, *dw, ws, h=h)  # noqa: E731
    new = lambda: (_nan(T, d), _nan(F, d), _nan(F, d), _nan(T, F))  # noqa: E731
    dx, dwg, dwu, again = new()
    back(dx, (dwg, dwu), again)
    one = new()
    back(one[0])
    back(None, one[1:3])
    back(h=one[3])
    for a, b in zip(one, (dx, dwg, dwu, again)):
        assert torch.equal(a, b)
    fws, out = tw.glu_packed_workspace(T, d, F), new()

    def step():
        tw.twell_glu_forward_packed(x, wg, wu, "silu", h, g, u, fws)
        back(out[0], out[1:3], out[3])

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in range(3):
        x.copy_(_rnd(T, d, seed=50 + n))
        graph.replay()
        got = [v.clone() for v in (h, g.code, g.scale, u.code, *out)]
        step()
        assert all(torch.equal(a, b) for a, b in zip(got, (h, g.code, g.scale, u.code, *out)))


def test_empty(gpu_lib):
    """No rows: nothing is done, weight gradients are zeros."""
    import torch
    tw = gpu_lib
    say("case act8 empty")
    p = tw.PackedAct.empty(0, 64)
    tw.twell_act_pack(_nan(0, 64), p)
    tw.twell_act_unpack(p, _nan(0, 64))
    x, w, h = _nan(0, 128), _rnd(64, 128), _nan(0, 64)
    tw.twell_glu_forward_packed(x, w, w, "silu", h, p, p)
    dwg, dwu = _nan(64, 128), _nan(64, 128)
    tw.twell_glu_backward_packed(x, w, w, p, p, h, "silu", None, dwg, dwu, tw.glu_backward_workspace(0, 128, 64, torch.bfloat16))
    assert not dwg.any() and not dwu.any()


def test_every_scale(gpu_lib):
    """Blocks whose largest is 127 steps of every mantissa of 8 bits, or next to that: the quotients that make the scale
    and its reciprocal are those of a division."""
    import torch
    say("case act pack, every scale")
    step = torch.arange(128, 256, device="cuda").float()
    tops = torch.cat([torch.nextafter(step * 127, torch.full_like(step, to)) for to in (0.0, math.inf)] + [step * 127])
    tops = torch.cat([tops * 2.0 ** e for e in (-90, -60, -31, -8, 0, 9, 50, 100)])
    x = _rnd(tops.numel(), 32, dtype="float32", seed=8).clamp(-3, 3) / 4 * tops[:, None]
    x[:, 7] = tops
    x[::2, 7] *= -1
    _check_pack(gpu_lib, x)
    _check_pack(gpu_lib, _rnd(20000, 64, dtype="float32", seed=9) * torch.exp2(_rnd(20000, 1, dtype="float32", scale=12)))
