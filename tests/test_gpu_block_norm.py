"""twell_block_norm_forward and _backward against their formulas in 64 bits,
element by element within the bounds of dense_ref.py."""

import itertools

import pytest

import dense_ref
from helpers import say

pytestmark = pytest.mark.gpu

EPS, ALPHA = 1e-5, 0.75


def _case(T, d, kind="rms", post=True, pre=True, block=True, bias=False, weights=True, span=0, r="float32", y="float32",
          n="float32", w="float32", dn="float32", seed=0, offset=0):
    """Device inputs; with an offset every tensor starts that many elements into its buffer."""
    import torch
    gen = torch.Generator().manual_seed(seed + T * 31 + d)
    dt = lambda name: getattr(torch, name)  # noqa: E731

    def rnd(*shape, dtype, scale=1.0, shift=0.0):
        n_el = 1
        for s in shape:
            n_el *= s
        buf = torch.zeros(n_el + offset, dtype=dt(dtype))
        buf[offset:] = (torch.randn(n_el, generator=gen) * scale + shift).to(dt(dtype))
        return buf.cuda()[offset:].view(shape)

    c = dict(T=T, d=d, kind=kind, post=post, pre=pre, span=span)
    c["res"] = rnd(T, d, dtype=r, scale=2.0)
    c["y"] = rnd(T, d, dtype=y, shift=0.3) if block else None
    c["gate"] = rnd(-(-T // span), d, dtype=r, shift=0.5) if span and block else None
    for k in ("post", "pre"):
        c["w_" + k] = rnd(d, dtype=w, scale=0.2, shift=1.0) if weights and c[k] else None
        c["b_" + k] = rnd(d, dtype=w, scale=0.2) if bias and c[k] else None
    c["dout"] = rnd(T, d, dtype=r, scale=0.1)
    c["dn"] = rnd(T, d, dtype=dn, scale=0.1) if pre else None
    c["new"] = lambda *shape, dtype: rnd(*shape, dtype=dtype).fill_(float("nan"))
    c["types"] = dict(r=r, y=y, n=n)
    return c


def _bn(tw, c):
    return tw.BlockNorm(c["kind"], EPS, ALPHA, c["post"], c["w_post"], c["b_post"], c["w_pre"], c["b_pre"])


def _forward(tw, c):
    T, d, t = c["T"], c["d"], c["types"]
    out = c["new"](T, d, dtype=t["r"]) if c["y"] is not None else None
    n = c["new"](T, d, dtype=t["n"]) if c["pre"] else None
    tw.twell_block_norm_forward(_bn(tw, c), c["res"], c["y"], out, n, gate=c["gate"], gate_span=c["span"])
    return {"out": out, "n": n}


def _backward(tw, c, dout=True):
    import torch
    T, d, t = c["T"], c["d"], c["types"]
    got = {"dres": c["new"](T, d, dtype=t["r"])}
    if c["y"] is not None:
        got["dy"] = c["new"](T, d, dtype=t["y"])
    if c["gate"] is not None:
        got["dgate"] = c["new"](*c["gate"].shape, dtype=t["r"])
    for k in ("w_post", "b_post") if c["post"] and c["y"] is not None else ():
        got["d" + k] = torch.full((d,), float("nan"), device="cuda")
    for k in ("w_pre", "b_pre") if c["pre"] else ():
        got["d" + k] = torch.full((d,), float("nan"), device="cuda")
    ws = tw.block_norm_workspace(T, d)
    ws.fill_(0xFF)  # NaN
    args = {k: got.get(k) for k in ("dgate", "dw_post", "db_post", "dw_pre", "db_pre")}
    tw.twell_block_norm_backward(_bn(tw, c), c["res"], c["y"], c["dout"] if dout else None, c["dn"], got["dres"],
                                 got.get("dy"), ws, gate=c["gate"], gate_span=c["span"], **args)
    return got


def _check(tw, c, dout=True):
    par = (c["w_post"], c["b_post"]), (c["w_pre"], c["b_pre"])
    rest = (c["kind"], EPS, ALPHA, c["post"] and c["y"] is not None, *par)
    want = dense_ref.norm_forward(c["res"], c["y"], c["gate"], c["span"], *rest)
    for k, got in _forward(tw, c).items():
        if got is not None:
            dense_ref.check(got, *_rounded(want[k], got), k)
    if dout or c["dn"] is not None:
        want = dense_ref.norm_backward(c["res"], c["y"], c["gate"], c["span"], c["dout"] if dout else None, c["dn"], *rest)
        for k, got in _backward(tw, c, dout).items():
            dense_ref.check(got, *_rounded(want[k], got), k)


def _rounded(pair, got):
    """The bound with the rounding to the stored type."""
    value, bound = pair
    return value, bound + dense_ref.half_step(value.abs() + bound, got.dtype)


SHAPES = [(1, 64), (5, 1), (3, 7), (2, 511), (9, 512), (4, 513), (7, 1001), (33, 1024), (6, 1032), (5, 2048), (3, 2056),
          (4, 4096), (2, 4104), (3, 8192), (2, 8191), (700, 96), (1025, 64), (1537, 40)]


@pytest.mark.parametrize("shape", SHAPES, ids=[f"T{t}_d{d}" for t, d in SHAPES])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_shapes(gpu_lib, shape, kind):
    say(f"case block norm {shape} {kind}")
    _check(gpu_lib, _case(*shape, kind=kind, bias=kind == "layer", span=2))


TYPES = list(itertools.product(["float32", "bfloat16"], repeat=4))


@pytest.mark.parametrize("types", TYPES, ids=["-".join(t[0] for t in c) for c in TYPES])
def test_types(gpu_lib, types):
    r, y, n, dn = types
    say(f"case block norm types {types}")
    for d, w in ((200, "float32"), (201, "bfloat16")):
        _check(gpu_lib, _case(21, d, r=r, y=y, n=n, dn=dn, w=w, span=4, bias=True))


@pytest.mark.parametrize("parts", list(itertools.product([False, True], repeat=4)))
def test_parts(gpu_lib, parts):
    """Every choice of the parts: a block, a norm after it, a norm before the next, weights."""
    block, post, pre, weights = parts
    say(f"case block norm parts {parts}")
    for span in (0, 3):
        for dout in (True, False):
            if not block and not pre:
                continue
            _check(gpu_lib, _case(17, 256, block=block, post=post, pre=pre, weights=weights, span=span), dout=dout)


@pytest.mark.parametrize("T,span", [(1, 1), (600, 1), (1200, 2), (1200, 3), (1200, 5), (1200, 599), (1200, 600),
                                    (1200, 1199), (1200, 1200), (1200, 5000), (513, 512), (514, 2), (4099, 7),
                                    (4099, 9), (4099, 64), (5000, 2500), (512, 512), (9000, 9000)])
def test_gate_spans(gpu_lib, T, span):
    """Gate rows that end inside, at and across the workgroups' rows."""
    say(f"case block norm T={T} span={span}")
    _check(gpu_lib, _case(T, 72, span=span))


@pytest.mark.parametrize("d", [1, 4, 15, 16, 17, 32, 33, 64, 100, 128, 129, 160, 256, 257])
@pytest.mark.parametrize("T,span", [(1, 0), (3, 1), (50, 3), (61, 16), (64, 64), (3000, 17), (4097, 1), (20011, 20011),
                                    (9001, 4500)])
def test_narrow_rows(gpu_lib, d, T, span):
    """Rows that share a wave: their own sums, columns past d, the last rows of a wave, gate rows that end inside one."""
    say(f"case block norm narrow T={T} d={d} span={span}")
    _check(gpu_lib, _case(T, d, kind="layer" if d % 3 else "rms", bias=T % 2 == 1, span=span, y="bfloat16"))


@pytest.mark.parametrize("offset", [1, 2, 8])
def test_alignment(gpu_lib, offset):
    say(f"case block norm offset {offset}")
    _check(gpu_lib, _case(11, 256, r="bfloat16", y="bfloat16", n="bfloat16", dn="bfloat16", span=2, offset=offset))


@pytest.mark.parametrize("d", [9, 15, 100, 511, 513, 519, 1001, 1025, 1031, 2049, 4100, 8191])
@pytest.mark.parametrize("post", [False, True])
def test_sum_in_place(gpu_lib, d, post):
    """out may be res: the same bits as with a tensor of its own."""
    import torch
    say(f"case block norm in place d={d} post={post}")
    c = _case(600, d, post=post, span=3)
    want = _forward(gpu_lib, c)
    out, n = c["res"].clone(), torch.empty_like(want["n"])
    gpu_lib.twell_block_norm_forward(_bn(gpu_lib, c), out, c["y"], out, n, gate=c["gate"], gate_span=3)
    assert torch.equal(out, want["out"]) and torch.equal(n, want["n"])


def test_rows_of_one_value(gpu_lib):
    """Rows without deviation, rows of zeros, and very large and small values stay finite and within the bounds."""
    import torch
    say("case block norm constant rows")
    for kind in ("rms", "layer"):
        c = _case(6, 384, kind=kind, span=1)
        for t in (c["res"], c["y"]):
            t[0] = 0.0
            t[1] = 3.0
            t[2] *= 1e-20
            t[3] *= 1e15
        c["gate"][0] = 0.0
        _check(gpu_lib, c)


def test_non_finite_row_stays_alone(gpu_lib):
    import torch
    say("case block norm non-finite row")
    c = _case(8, 256, span=1)
    good = _forward(gpu_lib, c)
    c["y"][3, 7] = float("nan")
    c["res"][5, 9] = float("inf")
    bad = _forward(gpu_lib, c)
    rows = [0, 1, 2, 4, 6, 7]
    for k in ("out", "n"):
        assert torch.equal(good[k][rows], bad[k][rows])
        assert not torch.isfinite(bad[k][3]).any() or k == "out"
        assert not torch.isfinite(bad[k][5, 9])


def test_same_bits_in_place_and_on_a_stream(gpu_lib):
    """Repeated calls, out over res, dres over dout, and a stream of its own give the same bits."""
    import torch
    say("case block norm same bits")
    c = _case(1300, 1000, span=300, r="bfloat16", n="bfloat16")
    first, grads = _forward(gpu_lib, c), _backward(gpu_lib, c)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        again, grads2 = _forward(gpu_lib, c), _backward(gpu_lib, c)
        torch.cuda.current_stream().synchronize()
    for a, b in ((first, again), (grads, grads2)):
        for k in a:
            assert torch.equal(a[k], b[k]), k
    res = c["res"].clone()
    gpu_lib.twell_block_norm_forward(_bn(gpu_lib, c), res, c["y"], res, again["n"], gate=c["gate"], gate_span=300)
    assert torch.equal(res, first["out"]) and torch.equal(again["n"], first["n"])


def test_no_rows(gpu_lib):
    """T = 0: nothing is written but the weights' gradients, which are 0."""
    import torch
    say("case block norm T=0")
    c = _case(0, 128)
    _forward(gpu_lib, c)
    got = _backward(gpu_lib, c)
    for k in ("dw_post", "db_post", "dw_pre", "db_pre"):
        assert not got[k].any(), k


def test_past_32_bits(gpu_lib):
    """Rows whose offset in elements does not fit 32 bits."""
    import torch
    T, d = (1 << 32) // 8192 + 3, 8192
    say(f"case block norm T={T} d={d}")
    res = torch.ones((T, d), dtype=torch.bfloat16, device="cuda")
    y = torch.full((T, d), 2.0, dtype=torch.bfloat16, device="cuda")
    res[-1] = 3.0
    bn = gpu_lib.BlockNorm("rms", 1e-6, 0.5, True)
    n = torch.zeros_like(res)
    gpu_lib.twell_block_norm_forward(bn, res, y, res, n)
    assert (res[-1] == 3.5).all() and (res[T - 4:T - 1] == 1.5).all() and (res[0] == 1.5).all()
    assert (n[-4:] == 1).all() and (n[0] == 1).all()


def test_refusals(gpu_lib):
    import torch
    tw = gpu_lib
    c = _case(4, 64, span=2)
    n = torch.empty_like(c["res"])
    f = lambda **k: tw.twell_block_norm_forward(  # noqa: E731
        *[k.get(a, v) for a, v in (("bn", _bn(tw, c)), ("res", c["res"]), ("y", c["y"]), ("out", n), ("n", n.clone()))],
        gate=k.get("gate", c["gate"]), gate_span=k.get("span", 2))
    f()
    for k, err in ((dict(y=c["y"][:2]), ValueError), (dict(out=n.bfloat16()), TypeError), (dict(gate=c["gate"][:1]), ValueError),
                   (dict(res=c["res"].t()), ValueError), (dict(span=0), ValueError), (dict(n=n.cpu()), ValueError),
                   (dict(res=c["res"].half()), TypeError), (dict(res=c["res"][:, :32].contiguous()), ValueError)):
        with pytest.raises(err):
            f(**k)
    with pytest.raises(ValueError):
        tw.BlockNorm("batch")
    with pytest.raises(tw.TwellError):
        f(out=None, n=None)
    with pytest.raises(tw.TwellError):
        tw.twell_block_norm_forward(tw.BlockNorm(eps=0.0), c["res"], None, None, n)
    wide = torch.zeros((1, 8200), device="cuda")
    with pytest.raises(tw.TwellError):
        tw.twell_block_norm_forward(tw.BlockNorm(), wide, None, None, wide.clone())
    with pytest.raises(tw.TwellError):  # a workspace that is too small
        tw.twell_block_norm_backward(tw.BlockNorm(), c["res"], None, c["dout"], c["dn"], n, None,
                                     torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):  # a workspace in host memory
        tw.twell_block_norm_backward(tw.BlockNorm(), c["res"], None, c["dout"], c["dn"], n, None,
                                     torch.empty(1 << 20, dtype=torch.uint8))
