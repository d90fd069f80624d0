"""twell_adamw_step and twell_adamw_unpack against a plain AdamW in 64 bits.

Bounds, from the arithmetic: a step's fp32 operations each round by at most
u = 2^-24, about six of them follow one another in m and v and ten in the
update, so m and v are within 8 u of their terms' magnitudes and p within 3 u of
p (the decay constant, its product, the sum) plus 16 u of the update's terms
(beta1 m and (1 - beta1) g may cancel); a bf16 p or copy adds half a step of
bf16, at most 2^-8.  An 8-bit state is one of the two codes around its value: relative steps of 2^-3
(m) and 2^-4 (sqrt(v)), plus the flush of values 2^-15 below the block's
largest."""

import numpy as np
import pytest

from helpers import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HYPER = dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, step=3)


def _plain(p, g, m, v, wd, lr, beta1, beta2, eps, step):
    m1 = beta1 * m + (1 - beta1) * g
    v1 = beta2 * v + (1 - beta2) * g * g
    upd = lr / (1 - beta1 ** step) * m1 / (np.sqrt(v1) / np.sqrt(1 - beta2 ** step) + eps)
    # the update's rounding errors scale with its terms, which may cancel in m
    terms = np.abs(upd) * (beta1 * np.abs(m) + (1 - beta1) * np.abs(g)) / np.maximum(np.abs(m1), 1e-300)
    return p * (1 - lr * wd) - upd, m1, v1, terms


def _tensors(sizes, bits, pdt, gdt, offset=0, seed=0, copy=True):
    """Device tensors (slices that start `offset` elements into their buffers) and their 64-bit values."""
    import torch
    gen = torch.Generator().manual_seed(seed)
    sets = []
    for i, n in enumerate(sizes):
        def new(dtype, fill=None):
            buf = torch.zeros(n + offset, dtype=dtype)
            t = buf[offset:]
            if fill is not None:
                t.copy_(fill)
            return buf.cuda()[offset:]
        t = dict(p=new(pdt, torch.randn(n, generator=gen)), grad=new(gdt, 0.1 * torch.randn(n, generator=gen)),
                 weight_decay=0.1 * (i % 2))
        if copy and pdt == torch.float32 and i % 3 != 2:
            t["copy"] = new(torch.bfloat16)
        blocks = -(-n // 256)
        if bits == 32:
            t.update(m=new(torch.float32, 0.05 * torch.randn(n, generator=gen)),
                     v=new(torch.float32, (0.1 * torch.randn(n, generator=gen)) ** 2))
        else:
            t.update(m=new(torch.uint8, torch.randint(0, 256, (n,), generator=gen)),
                     v=new(torch.uint8, torch.randint(0, 256, (n,), generator=gen)),
                     m_scale=0.05 + torch.rand(blocks, generator=gen).cuda(),
                     v_scale=0.05 + torch.rand(blocks, generator=gen).cuda(),
                     m_values=new(torch.float32), v_values=new(torch.float32))
        sets.append(t)
    return sets


def _decode(code, scale, signed):
    """The values of codes, from their definition: mantissa steps of an octave below the scale."""
    code = code.astype(np.int64)
    mag = code & 127 if signed else code
    per, top = (8, 127) if signed else (16, 255)
    steps = top - mag  # steps below 1.0; an octave below 1 runs from 0.5 to 1 in `per` equal steps
    octave = -(-steps // per)
    val = np.where(mag == 0, 0.0, 2.0 ** -octave * (1 + (octave * per - steps) / per))
    val = np.where(signed & (code > 127), -val, val)
    return val * np.repeat(scale.astype(np.float64), 256)[: code.size]


def _host(t, k):
    return None if t.get(k) is None else t[k].double().cpu().numpy() if t[k].is_floating_point() else t[k].cpu().numpy()


def _state(t, bits):
    if bits == 32:
        return _host(t, "m"), _host(t, "v")
    return (_decode(_host(t, "m"), _host(t, "m_scale"), True), _decode(_host(t, "v"), _host(t, "v_scale"), False) ** 2)


def _step(tw, sets, **kw):
    import torch
    h = dict(HYPER, **kw)
    params = tw.AdamWTensors(sets)
    tw.twell_adamw_step(params, h["lr"], h["beta1"], h["beta2"], h["eps"], h["step"], seed=h.get("seed", 11),
                        grad_scale=h.get("grad_scale"))
    if params.can_unpack:
        tw.twell_adamw_unpack(params)
    torch.cuda.synchronize()


def _check(sets, before, bits, pdt, clip=1.0):
    import torch
    for i, (t, (p0, g, m0, v0)) in enumerate(zip(sets, before)):
        n = p0.size
        if n == 0:
            continue
        h = {k: HYPER[k] for k in ("lr", "beta1", "beta2", "eps", "step")}
        p, m, v, upd = _plain(p0, g * clip, m0, v0, t["weight_decay"], **h)
        tol = 3 * U * np.abs(p0) + 16 * U * upd + 4e-45
        if pdt == torch.bfloat16:
            tol = tol + 2.0 ** -8 * (np.abs(p) + tol)
        got = _host(t, "p")
        assert (np.abs(got - p) <= tol).all(), f"tensor {i} (n={n}): p off by {np.max(np.abs(got - p) / tol):.3g} bounds"
        if t.get("copy") is not None:
            assert torch.equal(t["copy"], t["p"].bfloat16()), f"tensor {i}: copy"
        if bits == 32:
            assert (np.abs(_host(t, "m") - m) <= 8 * U * (np.abs(0.9 * m0) + np.abs(0.1 * g * clip)) + 1e-40).all()
            assert (np.abs(_host(t, "v") - v) <= 8 * U * v + 1e-40).all()
            continue
        mc, rc = _decode(_host(t, "m"), _host(t, "m_scale"), True), _decode(_host(t, "v"), _host(t, "v_scale"), False)
        np.testing.assert_allclose(_host(t, "m_values"), mc, rtol=2 * U, err_msg="unpacked m")
        np.testing.assert_allclose(_host(t, "v_values"), rc * rc, rtol=4 * U, err_msg="unpacked v")
        top = lambda a: np.repeat([np.max(np.abs(a[b:b + 256])) for b in range(0, n, 256)], 256)[:n]  # noqa: E731
        assert (np.abs(mc - m) <= 2.0 ** -3 * np.abs(m) * (1 + 1e-5) + 2.0 ** -15 * top(m)).all(), f"tensor {i}: m codes"
        r = np.sqrt(v)
        assert (np.abs(rc - r) <= 2.0 ** -4 * r * (1 + 1e-5) + 2.0 ** -15 * top(r)).all(), f"tensor {i}: v codes"
        assert (rc[r > 1e-30] > 0).all(), "a root above 0 stays above 0"


SIZES = [1, 0, 7, 255, 256, 257, 2048, 8191, 8192, 8193, 20011]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pdt", ["float32", "bfloat16"])
@pytest.mark.parametrize("gdt", ["float32", "bfloat16"])
@pytest.mark.parametrize("offset", [0, 1, 8])
def test_adamw_step(gpu_lib, bits, pdt, gdt, offset):
    import torch
    pdt, gdt = getattr(torch, pdt), getattr(torch, gdt)
    say(f"case adamw {bits} {pdt} {gdt} offset {offset}")
    sets = _tensors(SIZES, bits, pdt, gdt, offset)
    before = [(_host(t, "p"), _host(t, "grad"), *_state(t, bits)) for t in sets]
    _step(gpu_lib, sets)
    _check(sets, before, bits, pdt)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_many_tensors_with_coefficient(gpu_lib, bits):
    """More tensors than one launch takes, gradients scaled by a value on the GPU, on a stream of its own."""
    import torch
    say(f"case adamw many tensors {bits}")
    sets = _tensors([(37 * i) % 3000 + 1 for i in range(131)], bits, torch.float32, torch.float32, seed=5)
    before = [(_host(t, "p"), _host(t, "grad"), *_state(t, bits)) for t in sets]
    clip = torch.full((1,), 0.25, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        _step(gpu_lib, sets, grad_scale=clip)
    _check(sets, before, bits, torch.float32, clip=0.25)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("offset", [0, 3])
def test_adamw_large_tensors(gpu_lib, bits, offset):
    """Enough elements for workgroups of several passes, ending inside a block, a wave's pair of blocks and a pass."""
    import torch
    say(f"case adamw large {bits} offset {offset}")
    sets = _tensors([2_000_003, 8192 * 5 + 256, 300_001], bits, torch.float32, torch.bfloat16, offset, seed=2)
    before = [(_host(t, "p"), _host(t, "grad"), *_state(t, bits)) for t in sets]
    _step(gpu_lib, sets)
    _check(sets, before, bits, torch.float32)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("bad", [0.0, float("inf"), float("-inf"), float("nan")])
def test_adamw_unusable_gradients_change_nothing(gpu_lib, bits, bad):
    import torch
    say(f"case adamw coefficient {bad}")
    sets = _tensors([300, 5], bits, torch.float32, torch.float32)
    keep = [{k: x.clone() for k, x in t.items() if hasattr(x, "clone") and not k.endswith("_values")} for t in sets]
    _step(gpu_lib, sets, grad_scale=torch.full((1,), bad, device="cuda"))
    for t, k in zip(sets, keep):
        for name, x in k.items():
            assert torch.equal(t[name], x), name


def test_adamw_non_finite_gradient(gpu_lib):
    """32 bits: only the element is lost; 8 bits: its block of 256 reads back as NaN."""
    import torch
    say("case adamw non-finite gradient")
    for bits in (32, 8):
        sets = _tensors([1000], bits, torch.float32, torch.float32, copy=False)
        sets[0]["grad"][300] = float("nan")
        sets[0]["grad"][700] = float("inf")
        _step(gpu_lib, sets)
        bad = torch.isnan(sets[0]["p"]).nonzero().flatten().tolist()
        assert bad == [300, 700], bad
        if bits == 8:
            lost = torch.isnan(sets[0]["m_values"])
            assert lost[256:768].all() and not lost[:256].any() and not lost[768:].any()


def test_adamw_8bit_rounding(gpu_lib):
    """The same seed gives the same bits, another seed others, and the codes' mean is the value: over 400 seeds the
    mean of a value rounded to one of two steps (at most 2^-3 of it apart) has a deviation below 2^-4 / 20 of it; five
    deviations are allowed."""
    import torch
    say("case adamw 8-bit rounding")
    n = 512
    gen = torch.Generator().manual_seed(9)
    grad = torch.rand(n, generator=gen).cuda() * 0.9 + 0.1
    total_m, total_r, first = np.zeros(n), np.zeros(n), None
    for seed in range(400):
        z = lambda dt: torch.zeros(n, dtype=dt, device="cuda")  # noqa: E731
        t = dict(p=z(torch.float32), grad=grad, m=z(torch.uint8), v=z(torch.uint8),
                 m_scale=torch.zeros(2, device="cuda"), v_scale=torch.zeros(2, device="cuda"))
        _step(gpu_lib, [t], seed=seed, step=1)
        if seed < 2:
            again = dict(t, **{k: torch.zeros_like(t[k]) for k in ("p", "m", "v", "m_scale", "v_scale")})
            _step(gpu_lib, [again], seed=0, step=1)
            same = torch.equal(again["m"], t["m"]) and torch.equal(again["v"], t["v"])
            assert same == (seed == 0)
        m, v = _state(t, 8)
        total_m += m
        total_r += np.sqrt(v)
    g = grad.double().cpu().numpy()
    for got, want in ((total_m / 400, 0.1 * g), (total_r / 400, np.sqrt(0.05) * g)):
        assert np.max(np.abs(got / want - 1)) < 5 * 2.0 ** -4 / 20


def test_adamw_past_32_bits(gpu_lib):
    """Elements whose index does not fit 32 bits."""
    import torch
    n = (1 << 32) + 5
    say("case adamw past 32 bits")
    t = dict(p=torch.ones(n, dtype=torch.bfloat16, device="cuda"), grad=torch.zeros(n, dtype=torch.bfloat16, device="cuda"),
             m=torch.zeros(n, dtype=torch.uint8, device="cuda"), v=torch.zeros(n, dtype=torch.uint8, device="cuda"),
             m_scale=torch.zeros(n // 256 + 1, device="cuda"), v_scale=torch.zeros(n // 256 + 1, device="cuda"))
    at = [0, 5, (1 << 31) + 3, (1 << 32) - 1, 1 << 32, n - 1]
    for i in at:
        t["grad"][i:i + 1].fill_(1.0)
    _step(gpu_lib, [t], lr=0.5, step=1)
    for i in at:
        assert t["p"][i].item() == 0.5 and t["m"][i].item() > 0 and t["v"][i].item() > 0
    assert sum(int((x != 1).sum()) for x in t["p"].split(1 << 30)) == len(at)
    assert sum(int((x != 0).sum()) for x in t["m"].split(1 << 30)) == len(at)


def test_adamw_refusals(gpu_lib):
    import torch
    tw = gpu_lib
    good = _tensors([64], 8, torch.float32, torch.float32)[0]
    for change, err in (({"m": None}, ValueError), ({"m_scale": None}, ValueError), ({"v": good["v"].float()}, TypeError),
                        ({"grad": good["grad"][:32]}, ValueError), ({"grad": good["grad"].cpu()}, ValueError),
                        ({"p": good["p"].half()}, TypeError), ({"grad": torch.zeros(128, device="cuda")[::2]}, ValueError),
                        ({"copy": good["p"].clone()}, TypeError)):
        with pytest.raises(err):
            tw.AdamWTensors([dict(good, **change)])
    params = tw.AdamWTensors([good])
    for bad in (dict(lr=-1.0), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=0.0), dict(step=0), dict(lr=float("nan"))):
        h = dict(HYPER, **bad)
        with pytest.raises(tw.TwellError):
            tw.twell_adamw_step(params, h["lr"], h["beta1"], h["beta2"], h["eps"], h["step"])
    with pytest.raises(ValueError):
        tw.twell_adamw_unpack(tw.AdamWTensors(_tensors([64], 32, torch.float32, torch.float32)))
    for scale in (torch.ones(1), torch.ones(2, device="cuda"), torch.ones(1, device="cuda", dtype=torch.float64)):
        with pytest.raises((ValueError, TypeError)):
            tw.twell_adamw_step(params, HYPER["lr"], HYPER["beta1"], HYPER["beta2"], HYPER["eps"], 1, grad_scale=scale)
