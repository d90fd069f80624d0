"""twell_logprob_forward and _backward against their formulas in 64 bits, element by
element within the bounds of tokens_ref.py."""

import math

import pytest

import tokens_ref
from helpers import say

pytestmark = pytest.mark.gpu

TYPES = ["bfloat16", "float32"]
INF, NAN = math.inf, math.nan


def _logits(T, V, dtype, seed=0, spread=3.0, ld=None):
    """Rows in a wider buffer, whose other elements are NaN."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.full((T, ld or V), NAN, device="cuda", dtype=getattr(torch, dtype))
    z[:, :V] = torch.randn((T, V), generator=gen, device="cuda") * spread
    return z[:, :V]


def _targets(T, V, dtype="int64", seed=0):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed + 77)
    return torch.randint(-1, V + 1, (T,), generator=gen, device="cuda").to(getattr(torch, dtype))


def _new(*shape):
    import torch
    return torch.full(shape, 7.25, device="cuda")


def _forward(tw, z, targets, scale=1.0, k=0, most=None):
    import torch
    T, V = z.shape
    got = {"norm": _new(T, 2), "entropy": _new(T), "logp": _new(T), "top_logp": _new(T, k) if k else None}
    idx = torch.full((T, k), -5, dtype=torch.int32, device="cuda") if k else None
    ws = tw.logprob_workspace(most or T, V, k)
    if ws is not None:
        ws.fill_(0xFF)
    tw.twell_logprob_forward(z, targets, got["logp"], got["norm"], ws, scale=scale, entropy=got["entropy"],
                             top_logp=got["top_logp"], top_idx=idx)
    return got, idx


def _check_forward(tw, z, targets, scale=1.0, k=0):
    import torch
    got, idx = _forward(tw, z, targets, scale, k)
    want, order = tokens_ref.logprob_forward(z, targets, scale, k)
    for name in ("norm", "entropy", "logp") + (("top_logp",) if k else ()):
        tokens_ref.check(got[name], *want[name], name)
    if k:
        assert torch.equal(idx.long(), order), "top_idx"
    return got


def _check_backward(tw, z, targets, scale=1.0, entropy=True, logp=True, in_place=False, seed=3):
    import torch
    T, V = z.shape
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dlogp, dent = (torch.randn(T, generator=gen, device="cuda") for _ in range(2))
    fwd, _ = _forward(tw, z, targets, scale)
    want, bound = tokens_ref.logprob_backward(z, targets, fwd["norm"], dlogp if logp else None, scale, fwd["entropy"],
                                              dent if entropy else None)
    if in_place:
        dz = z
    else:
        wide = torch.full((T, V + 3), 7.25, dtype=z.dtype, device="cuda")
        dz = wide[:, :V]
    tw.twell_logprob_backward(z, targets if logp else None, fwd["norm"], dlogp if logp else None, dz, scale=scale,
                              entropy=fwd["entropy"] if entropy else None, dentropy=dent if entropy else None)
    if not in_place:
        assert (wide[:, V:] == 7.25).all()
    tokens_ref.check(dz, want, bound, "dlogits")


# widths around the pieces of 4 and 8, the workgroup's 256 threads, segments of 4096 and rows of 48 KB, which few rows are not cut below
WIDTHS = [1, 2, 3, 4, 5, 7, 8, 9, 63, 255, 257, 500, 537, 944, 1000, 2047, 2048, 2049, 4096, 4097, 8191, 8200, 12288, 12289, 20001, 24576, 24577, 50001]


@pytest.mark.parametrize("V", WIDTHS)
@pytest.mark.parametrize("dtype", TYPES)
def test_widths(gpu_lib, V, dtype):
    say(f"case logprob V={V} {dtype}")
    for T in (1, 3):
        for k in sorted({0, 1, min(V, 5), min(V, 64)}):
            _check_forward(gpu_lib, _logits(T, V, dtype, seed=V + k), _targets(T, V, seed=k), 0.8, k)
        _check_backward(gpu_lib, _logits(T, V, dtype, seed=V), _targets(T, V), 0.8)


@pytest.mark.parametrize("T,V", [(1, 131072), (2, 262145), (17, 30000), (100, 9000), (341, 12289), (400, 26000), (1023, 25001), (1024, 8192), (1025, 4100),
                                 (3000, 515)])
@pytest.mark.parametrize("dtype", TYPES)
def test_rows(gpu_lib, T, V, dtype):
    say(f"case logprob T={T} V={V} {dtype}")
    z, t = _logits(T, V, dtype, seed=T), _targets(T, V, "int32")
    _check_forward(gpu_lib, z, t, 1.25, 20)
    _check_forward(gpu_lib, z, t)
    _check_backward(gpu_lib, z, t, 1.25)


@pytest.mark.parametrize("extra", [1, 2, 3, 5, 8, 64])
@pytest.mark.parametrize("dtype", TYPES)
def test_strided_rows(gpu_lib, extra, dtype):
    """Rows of a wider buffer, at any alignment of their elements, and the gradient in their place."""
    import torch
    T, V = 9, 25003
    say(f"case logprob strided {extra} {dtype}")
    z, t = _logits(T, V, dtype, ld=V + extra), _targets(T, V)
    _check_forward(gpu_lib, z, t, 1.0, 7)
    _check_forward(gpu_lib, z[:, 1:], t, 1.0, 7)
    _check_backward(gpu_lib, z, t)
    whole = z.as_strided((T, V + extra), (V + extra, 1))
    _check_backward(gpu_lib, z, t, in_place=True)
    assert torch.isnan(whole[:, V:]).all()


@pytest.mark.parametrize("spread", [0.01, 30.0, 1000.0])
@pytest.mark.parametrize("dtype", TYPES)
def test_flat_and_peaked_rows(gpu_lib, spread, dtype):
    say(f"case logprob spread {spread} {dtype}")
    for T, V in ((2, 6001), (2, 30001), (1100, 6001)):
        z, t = _logits(T, V, dtype, spread=spread), _targets(T, V)
        z[0] += 1e4
        _check_forward(gpu_lib, z, t, 1.0, 12)
        _check_backward(gpu_lib, z, t)


@pytest.mark.parametrize("order", ["up", "down"])
@pytest.mark.parametrize("dtype", TYPES)
def test_sorted_rows(gpu_lib, order, dtype):
    """The maximum rises with every piece, or never."""
    import torch
    say(f"case logprob sorted {order} {dtype}")
    for T, V in ((2, 40000), (2, 9001), (1030, 9001)):
        z, t = _logits(T, V, dtype), _targets(T, V)
        z.copy_(torch.sort(z, dim=1, descending=order == "down").values)
        _check_forward(gpu_lib, z, t, 1.0, 64)
        _check_backward(gpu_lib, z, t)


@pytest.mark.parametrize("T,V", [(2, 9001), (2, 31001), (1100, 9001)])
@pytest.mark.parametrize("dtype", TYPES)
def test_equal_logits(gpu_lib, T, V, dtype):
    """Equal logits in bulk: the lowest indices first, +0 and -0 the same value."""
    say(f"case logprob equal logits T={T} V={V} {dtype}")
    t = _targets(T, V)
    z = _logits(T, V, dtype)
    z.zero_()
    z[:, 1::3] *= -1
    got = _check_forward(gpu_lib, z, t, 1.0, 33)
    assert abs(float(got["entropy"][0]) - math.log(V)) < 1e-4
    z[:, 5000:8000] = 1  # more than the list of candidates holds
    z[:, 8500] = 2
    _check_forward(gpu_lib, z, t, 1.0, 64)
    z[:, ::2] = -1
    _check_forward(gpu_lib, z, t, 2.0, 40)
    _check_backward(gpu_lib, z, t)
    for few in (1, 5, 150, 250, 700):  # around the number from which on equal ones are told apart
        z.fill_(-3)
        z[:, 4000:4000 + few] = 5
        z[:, 4000 + few // 2] = 6
        for k in (1, 20, 64):
            _check_forward(gpu_lib, z, t, 1.0, k)


@pytest.mark.parametrize("T", [2, 1100])
@pytest.mark.parametrize("dtype", TYPES)
def test_all_in_few_threads(gpu_lib, T, dtype):
    """The largest logits lie where one thread reads them, more than the list of candidates holds among them."""
    import torch
    say(f"case logprob all in few threads T={T} {dtype}")
    V, E = 300000 if T == 2 else 60000, 8 if dtype == "bfloat16" else 4
    z, t = _logits(T, V, dtype), _targets(T, V)
    piece = torch.arange(V, device="cuda") // E % 256
    for thread, k in ((0, 64), (77, 20), (255, 33)):
        x = torch.where(piece == thread, z * 0.25 + 40, z)
        _check_forward(gpu_lib, x, t, 1.0, k)


SHORT = [(5, 1), (5, 9), (3, 511), (6, 517), (7, 1027), (5, 1028), (5, 2047), (5, 2055), (5, 2056), (2049, 2050), (2051, 4103), (2050, 4104)]


@pytest.mark.parametrize("T,V", SHORT)
@pytest.mark.parametrize("dtype", TYPES)
def test_short_rows(gpu_lib, T, V, dtype):
    """Rows that a wave holds in registers, up to the widths from which on a workgroup takes one; as they are,
    of few values, masked, and with the largest logits in few lanes."""
    import torch
    say(f"case logprob short rows T={T} V={V} {dtype}")
    E = 8 if dtype == "bfloat16" else 4
    z, t = _logits(T, V, dtype, seed=V, ld=V + 3), _targets(T, V)
    lane = torch.arange(V, device="cuda") // E % 64
    gen = torch.Generator(device="cuda").manual_seed(V)
    few = torch.randint(0, 3, (T, V), generator=gen, device="cuda").to(z.dtype)
    some = torch.where(torch.rand((T, V), generator=gen, device="cuda") < 0.98, -INF, z)
    none = some.clone()
    none[T // 2] = -INF
    for k in sorted({0, 1, min(V, 20), min(V, 24), min(V, 25), min(V, 64)}):
        _check_forward(gpu_lib, z, t, 0.7, k)
        if k:
            _check_forward(gpu_lib, few, t, 1.0, k)
            _check_forward(gpu_lib, torch.full_like(few, -2), t, 1.0, k)
            _check_forward(gpu_lib, some, t, 1.0, k)
            _check_forward(gpu_lib, none, t, 1.0, k)
            for lanes in (1, 5, 18):
                _check_forward(gpu_lib, torch.where(lane < lanes, z * 0.25 + 40, z), t, 1.0, k)
                _check_forward(gpu_lib, torch.where(lane < lanes, torch.round(z) + 40, few), t, 1.0, k)
    _check_backward(gpu_lib, z, t, 0.7)


@pytest.mark.parametrize("bad", [NAN, -NAN, INF])
@pytest.mark.parametrize("T,V", [(6, 700), (2049, 4099)])
@pytest.mark.parametrize("dtype", TYPES)
def test_nan_in_short_rows(gpu_lib, bad, T, V, dtype):
    """They spoil their own row, and no other that the same workgroup has."""
    import torch
    k = 6
    say(f"case logprob bad {bad} T={T} V={V} {dtype}")
    z, t = _logits(T, V, dtype), _targets(T, V).clamp(0, V - 1)
    clean, order = _forward(gpu_lib, z, t, 1.0, k)
    for where in (0, V // 2, V - 1):
        x = z.clone()
        x[1, where] = bad
        got, idx = _forward(gpu_lib, x, t, 1.0, k)
        rest = torch.arange(T, device="cuda") != 1
        for name, v in got.items():
            assert torch.isnan(v[1]).all(), name
            assert torch.equal(v[rest], clean[name][rest]), name
        assert idx[1].tolist() == list(range(k)) and torch.equal(idx[rest], order[rest])


@pytest.mark.parametrize("T,V", [(5, 700), (5, 2055), (2049, 3001), (2047, 3001)])
@pytest.mark.parametrize("dtype", TYPES)
def test_same_bits_with_any_alternatives(gpu_lib, T, V, dtype):
    """A row's sums do not depend on how many alternatives are asked for, nor on the run."""
    import torch
    say(f"case logprob bits T={T} V={V} {dtype}")
    z, t = _logits(T, V, dtype), _targets(T, V)
    one, _ = _forward(gpu_lib, z, t, 1.0, 0)
    for k in (0, 1, 20, 64, 64):
        got, idx = _forward(gpu_lib, z, t, 1.0, k)
        for name in ("norm", "entropy", "logp"):
            assert torch.equal(got[name], one[name]), (name, k)
    again, order = _forward(gpu_lib, z, t, 1.0, 64)
    assert torch.equal(again["top_logp"], got["top_logp"]) and torch.equal(order, idx)


@pytest.mark.parametrize("T,V", [(3, 8209), (3, 30011), (1100, 8209)])
@pytest.mark.parametrize("dtype", TYPES)
def test_masked_logits(gpu_lib, T, V, dtype):
    """-inf and the type's lowest value: parts of a row, all but one, all."""
    import torch
    say(f"case logprob masked T={T} V={V} {dtype}")
    k = 10
    for blank in (-INF, float(torch.finfo(getattr(torch, dtype)).min)):
        z, t = _logits(T, V, dtype), _targets(T, V)
        z[:, 100:7000] = blank
        t[2] = 150
        z[1] = blank
        z[0] = blank
        z[0, 77] = -3
        got = _check_forward(gpu_lib, z, t, 1.0, k)
        _check_backward(gpu_lib, z, t)
        _check_backward(gpu_lib, z, t, logp=False)
        if blank == -INF:
            assert got["norm"][1].tolist() == [-INF, 0] and got["entropy"][1] == 0
        else:  # nothing but equal values: as likely as each other
            assert abs(float(got["entropy"][1]) - math.log(V)) < 1e-4
        z.fill_(blank)
        _check_forward(gpu_lib, z, t, 1.0, k)
        _check_backward(gpu_lib, z, t)


@pytest.mark.parametrize("bad", [NAN, -NAN, INF])
@pytest.mark.parametrize("T,V", [(4, 8197), (4, 31013), (1100, 8197)])
@pytest.mark.parametrize("dtype", TYPES)
def test_nan_and_infinity(gpu_lib, bad, T, V, dtype):
    """They spoil their own row, wherever they stand in it."""
    import torch
    k = 6
    say(f"case logprob bad {bad} T={T} V={V} {dtype}")
    z, t = _logits(T, V, dtype), _targets(T, V).clamp(0, V - 1)
    clean, _ = _forward(gpu_lib, z, t, 1.0, k)
    for where in (0, 4095, 5000, V - 1):
        x = z.clone()
        x[1, where] = bad
        got, idx = _forward(gpu_lib, x, t, 1.0, k)
        for name, v in got.items():
            assert torch.isnan(v[1]).all(), name
            for r in (0, 2, T - 1):
                assert torch.equal(v[r], clean[name][r]), name
        assert idx[1].tolist() == list(range(k))
        dz = torch.zeros_like(x)
        gpu_lib.twell_logprob_backward(x, t, got["norm"], torch.ones(T, device="cuda"), dz)
        assert torch.isnan(dz[1]).all() and torch.isfinite(dz[0]).all() and torch.isfinite(dz[2:]).all()
        x[1, :] = -INF
        x[1, where] = NAN
        got, _ = _forward(gpu_lib, x, t, 1.0, k)
        assert torch.isnan(got["norm"][1]).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_parts_of_the_results(gpu_lib, dtype):
    """Every output by itself has the bits that it has with the others."""
    import torch
    tw = gpu_lib
    say(f"case logprob parts {dtype}")
    for T, V in ((3, 9000), (1100, 9000), (3, 30000)):
        k = 5
        z, t = _logits(T, V, dtype), _targets(T, V)
        all_, idx = _forward(tw, z, t, 1.0, k)
        ws = tw.logprob_workspace(T, V, k)
        a, b, c, d = _new(T), _new(T, 2), _new(T), _new(T, k)
        i = torch.empty_like(idx)
        tw.twell_logprob_forward(z, t, a, None, ws)
        tw.twell_logprob_forward(z, None, None, b, ws)
        tw.twell_logprob_forward(z, None, None, None, ws, entropy=c)
        tw.twell_logprob_forward(z, None, None, None, ws, top_logp=d, top_idx=i)
        for got, name in ((a, "logp"), (b, "norm"), (c, "entropy"), (d, "top_logp")):
            assert torch.equal(got, all_[name]), name
        assert torch.equal(i, idx)
        for parts in (dict(entropy=False), dict(logp=False)):
            _check_backward(tw, z, t, **parts)
        with pytest.raises(tw.TwellError):
            tw.twell_logprob_forward(z, None, None, None, ws)
    with pytest.raises(tw.TwellError):
        tw.twell_logprob_forward(z[:3], t[:3], _new(3), None)  # cut rows need the workspace


def test_targets_past_32_bits(gpu_lib):
    import torch
    say("case logprob, targets past 32 bits")
    z = _logits(4, 50, "float32")
    t = torch.tensor([3, 3 + (1 << 32), -(1 << 63), 50], device="cuda")
    got = _check_forward(gpu_lib, z, t)
    assert got["logp"][0] != 0 and not got["logp"][1:].any()
    _check_backward(gpu_lib, z, t)


def test_rows_past_32_bits(gpu_lib):
    """Rows whose offset does not fit 32 bits."""
    import torch
    T, V = 40, 1 << 26
    say("case logprob, logits of 2.7e9 elements")
    z = torch.zeros((T, V), dtype=torch.bfloat16, device="cuda")
    z[T - 1, V - 5], z[T - 1, V - 9] = 30, 29
    t = torch.full((T,), V - 5, device="cuda")
    got, idx = _forward(gpu_lib, z, t, 1.0, 2)
    assert idx[T - 1].tolist() == [V - 5, V - 9]
    tokens_ref.check(got["logp"][-1:], *[x[-1:] for x in tokens_ref.logprob_forward(z[-1:], t[-1:], 1.0)[0]["logp"]], "logp")
    gpu_lib.twell_logprob_backward(z, t, got["norm"], torch.ones(T, device="cuda"), z)
    assert float(z[T - 1, V - 9]) < -0.2 and float(z[T - 1, V - 5]) > 0.2


@pytest.mark.parametrize("dtype,bits", [("bfloat16", "int32"), ("float32", "int64")])
def test_more_rows_than_a_launch_has(gpu_lib, dtype, bits):
    """2^24 + 3 short rows: a workgroup of 256 threads each passes what a launch counts in 32 bits."""
    import torch
    T, V = (1 << 24) + 3, 3
    say(f"case logprob, {T} rows of {V} {dtype}")
    z, t = _logits(T, V, dtype, ld=4), _targets(T, V, bits)
    got, idx = _forward(gpu_lib, z, t, 0.5, 2)
    dz = torch.full((T, V), NAN, dtype=z.dtype, device="cuda")
    gpu_lib.twell_logprob_backward(z, t, got["norm"], got["logp"], dz, scale=0.5, entropy=got["entropy"],
                                   dentropy=got["entropy"])
    for some in (slice(0, 1000), slice(T - 1003, T)):
        want, order = tokens_ref.logprob_forward(z[some], t[some], 0.5, 2)
        for name in got:
            tokens_ref.check(got[name][some], *want[name], name)
        assert torch.equal(idx[some].long(), order), "top_idx"
        one = {name: x[some].contiguous() for name, x in got.items()}
        part = torch.empty_like(dz[some])
        gpu_lib.twell_logprob_backward(z[some], t[some].contiguous(), one["norm"], one["logp"], part, scale=0.5,
                                       entropy=one["entropy"], dentropy=one["entropy"])
        assert torch.equal(dz[some], part), "dlogits"
    assert bool((got["entropy"] < 1.1).all()) and not bool(dz.isnan().any())  # (ln 3 at most): every row is written


@pytest.mark.parametrize("T,V", [(1, 40000), (60, 9000), (1200, 3001)])
def test_same_bits_graph_and_streams(gpu_lib, T, V):
    """Repeated calls, a workspace for more rows, another stream and a captured graph's replays, the gradient in place
    among them, give the same bits."""
    import torch
    tw, k = gpu_lib, 9
    say(f"case logprob graph T={T} V={V}")
    z, t = _logits(T, V, "bfloat16"), _targets(T, V)
    src = z.clone()
    ws = tw.logprob_workspace(T + 100, V, k)
    logp, norm, ent, top = _new(T), _new(T, 2), _new(T), _new(T, k)
    idx = torch.empty((T, k), dtype=torch.int32, device="cuda")
    dlogp = torch.linspace(-1, 1, T, device="cuda")

    def step(stream=None):
        tw.twell_logprob_forward(z, t, logp, norm, ws, entropy=ent, top_logp=top, top_idx=idx, stream=stream)
        tw.twell_logprob_backward(z, t, norm, dlogp, z, entropy=ent, dentropy=dlogp, stream=stream)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in range(3):
        src.copy_(_logits(T, V, "bfloat16", seed=n))
        t.copy_(_targets(T, V, seed=n))
        want = None
        for how in ("eager", "graph", "side", "graph"):
            z.copy_(src)
            if ws is not None:
                ws.fill_(0xFF)
            if how == "graph":
                graph.replay()
            elif how == "side":
                side = torch.cuda.Stream()
                side.wait_stream(torch.cuda.current_stream())
                step(stream=side)
                side.synchronize()
            else:
                step()
            got = [v.clone() for v in (z, logp, norm, ent, top, idx)]
            want = want or got
            assert all(torch.equal(a, b) for a, b in zip(got, want)), how
