"""twell_embed_forward and _backward against their formulas in 64 bits, element by
element within the bounds of tokens_ref.py."""

import math

import pytest

import tokens_ref
from helpers import say

pytestmark = pytest.mark.gpu

TYPES = ["bfloat16", "float32"]


def _rnd(*shape, dtype="float32", seed=0, scale=1.0):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(getattr(torch, dtype))


def _ids(T, V, dtype="int64", seed=0, spread="uniform"):
    """uniform: some below 0 and some past V; text: a few ids have most of the tokens; one: all the same."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed + 1000)
    if spread == "one":
        t = torch.full((T,), V // 2, device="cuda")
    elif spread == "text":
        t = torch.exp(torch.rand(T, generator=gen, device="cuda", dtype=torch.float64) * math.log(V + 1)).long() - 1
    else:
        t = torch.randint(-max(1, V // 8), V + max(1, V // 8), (T,), generator=gen, device="cuda")
    return t.to(getattr(torch, dtype))


def _forward(tw, ids, table, out_type, scale):
    import torch
    out = torch.full((ids.shape[0], table.shape[1]), float("nan"), dtype=getattr(torch, out_type), device="cuda")
    tw.twell_embed_forward(ids, table, out, scale=scale)
    return out


def _check_forward(tw, ids, table, out_type, scale=1.0):
    got = _forward(tw, ids, table, out_type, scale)
    value, bound = tokens_ref.embed_forward(ids, table, scale)
    tokens_ref.check(got, value, bound, "out")


SHAPES = [(1, 1, 1), (1, 300, 2048), (2, 7, 3), (5, 9, 4), (33, 100, 5), (64, 3, 8), (100, 50, 7), (257, 1000, 17), (1000, 333, 96),
          (1003, 64, 1001), (4097, 2000, 40)]


@pytest.mark.parametrize("shape", SHAPES, ids=["T%d_V%d_d%d" % s for s in SHAPES])
@pytest.mark.parametrize("table", TYPES)
@pytest.mark.parametrize("out", TYPES)
def test_forward(gpu_lib, shape, table, out):
    say(f"case embed forward {shape} {table} {out}")
    T, V, d = shape
    rows = _rnd(V, d, dtype=table, seed=T)
    _check_forward(gpu_lib, _ids(T, V, seed=d), rows, out, 1.75)
    _check_forward(gpu_lib, _ids(T, V, "int32", seed=d), rows, out)


def test_forward_ids_past_32_bits(gpu_lib):
    """An id of 64 bits whose lower half is one of the table's rows is none of them."""
    import torch
    say("case embed forward, ids past 32 bits")
    table = _rnd(8, 16)
    ids = torch.tensor([3, 3 + (1 << 32), 3 - (1 << 32), (1 << 63) - 1, -(1 << 63), 7, 8, -1], device="cuda")
    got = _forward(gpu_lib, ids, table, "float32", 1.0)
    want = torch.zeros_like(got)
    want[0], want[5] = table[3], table[7]
    assert torch.equal(got, want)


def test_a_table_past_32_bits(gpu_lib):
    """Rows whose offset does not fit 32 bits, read, and written by the gradient."""
    import torch
    V, d = 1100000, 2048
    say("case embed, a table of 2.25e9 elements")
    table = torch.zeros((V, d), dtype=torch.bfloat16, device="cuda")
    last = _rnd(2, d, dtype="bfloat16", seed=3)
    table[-2:] = last
    ids = torch.tensor([V - 1, 0, V - 2], device="cuda")
    got = _forward(gpu_lib, ids, table, "bfloat16", 1.0)
    assert torch.equal(got, torch.stack((last[1], torch.zeros_like(last[0]), last[0])))
    table.fill_(1)
    gpu_lib.twell_embed_backward(ids, got, table, gpu_lib.embed_workspace(3, V, d))
    assert torch.equal(table[-2:], last) and int(table[:-2].count_nonzero()) == 0


def _backward(tw, ids, dout, start, accumulate, scale, most=None):
    """The gradient in a tensor that starts as `start`, with what lies before and behind it."""
    import torch
    V, d = start.shape
    around = torch.full((V * d + 2 * 64,), 3.0, dtype=start.dtype, device="cuda")
    table = around[64:64 + V * d].view(V, d)
    table.copy_(start)
    ws = tw.embed_workspace(most or ids.shape[0], V, d)
    ws.fill_(0xFF)
    tw.twell_embed_backward(ids, dout, table, ws, scale=scale, accumulate=accumulate)
    assert (around[:64] == 3).all() and (around[64 + V * d:] == 3).all()
    return table


def _check_backward(tw, ids, dout, V, table, accumulate, scale=1.0):
    import torch
    d = dout.shape[1]
    start = _rnd(V, d, dtype=table, seed=5) if accumulate else torch.full((V, d), float("nan"), device="cuda").to(getattr(torch, table))
    got = _backward(tw, ids, dout, start, accumulate, scale)
    value, bound = tokens_ref.embed_backward(ids, dout, V, scale, start if accumulate else None)
    tokens_ref.check(got, value, bound, "dtable")
    touched = torch.zeros(V, dtype=torch.bool, device="cuda")
    touched[ids[(ids >= 0) & (ids < V)].long()] = True
    if accumulate:
        assert torch.equal(got[~touched], start[~touched])
    else:
        assert not got[~touched].any()
    return got


# around the 1024 tokens, and 4096 slices of 256 columns of them, that one launch takes, the windows of 8 and 32, the counted ranks' 8192 tokens and the sorting
# passes' digits of 9 bits; widths around a workgroup's zeros
BACK = [(255, 3, 8), (256, 300, 260), (256, 5000, 3), (257, 40, 8), (200, 2, 17000), (40, 9000, 1000), (7, 700000, 12), (1024, 40, 1024), (1024, 40, 1028), (1024, 700, 250),
        (1025, 40, 8), (63, 900, 16400), (2048, 30, 8),
        (2049, 30, 8), (1, 1, 1), (1, 5, 64), (2, 3, 4), (31, 4, 5), (32, 1, 8), (33, 2, 3), (64, 5, 17), (65, 1, 1), (100, 1000, 96), (1000, 7, 33),
        (1003, 500, 1001), (8192, 600, 12), (8193, 511, 8), (8200, 512, 4), (20000, 100, 2), (30000, 70000, 20), (70000, 3, 5),
        (132000, 513, 4)]


@pytest.mark.parametrize("shape", BACK, ids=["T%d_V%d_d%d" % s for s in BACK])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("spread", ["uniform", "text", "one"])
def test_backward(gpu_lib, shape, accumulate, spread):
    T, V, d = shape
    say(f"case embed backward {shape} {spread} accumulate={accumulate}")
    _check_backward(gpu_lib, _ids(T, V, seed=T, spread=spread), _rnd(T, d, seed=d), V, "float32", accumulate, 0.75)


@pytest.mark.parametrize("dout", TYPES)
@pytest.mark.parametrize("table", TYPES)
@pytest.mark.parametrize("d", [1, 3, 4, 7, 8, 9, 40, 257])
def test_backward_types(gpu_lib, dout, table, d):
    say(f"case embed backward {dout} {table} d={d}")
    rows = _rnd(700, d, dtype=dout, seed=d)
    for accumulate in (False, True):
        for ids in ("int32", "int64"):
            _check_backward(gpu_lib, _ids(700, 90, ids, seed=d, spread="text"), rows, 90, table, accumulate, 1.5)


@pytest.mark.parametrize("T", [9000, 40000])
def test_backward_large_vocabulary(gpu_lib, T):
    """Keys of 28 bits: four sorting passes."""
    import torch
    V, d = (1 << 27) + 5, 3
    say(f"case embed backward V={V} T={T}")
    gen = torch.Generator(device="cuda").manual_seed(T)
    few = torch.randint(-5, V + 5, (T // 3,), generator=gen, device="cuda")
    few[:3] = torch.tensor([0, V - 1, V], device="cuda")
    ids = few[torch.randint(0, T // 3, (T,), generator=gen, device="cuda")]
    dout, table = _rnd(T, d), torch.zeros((V, d), device="cuda")
    gpu_lib.twell_embed_backward(ids, dout, table, gpu_lib.embed_workspace(T, V, d), accumulate=True)
    names, at = torch.unique(ids, return_inverse=True)
    value, bound = tokens_ref.embed_backward(at, dout, names.numel(), 1.0)
    real = (names >= 0) & (names < V)
    tokens_ref.check(table[names[real]], value[real], bound[real], "dtable")
    table[names[real]] = 0
    assert not table.any()


@pytest.mark.parametrize("T", [0, 5, 9000])
def test_backward_without_ids(gpu_lib, T):
    """No token, or only padding: zeros, or nothing is changed."""
    import torch
    say(f"case embed backward, T={T}, no ids")
    ids, dout = torch.full((T,), -1, device="cuda"), _rnd(T, 6)
    for accumulate in (False, True):
        start = _rnd(11, 6, seed=1)
        got = _backward(gpu_lib, ids, dout, start, accumulate, 1.0)
        assert torch.equal(got, start if accumulate else torch.zeros_like(start))


def test_padding_s_rows_are_not_read(gpu_lib):
    """NaN in the gradient of a padded token reaches no row."""
    import torch
    say("case embed backward, NaN in padded rows")
    ids = _ids(500, 40, seed=2)
    dout = _rnd(500, 24)
    dout[(ids < 0) | (ids >= 40)] = float("nan")
    _check_backward(gpu_lib, ids, torch.where(torch.isnan(dout), 0.0, dout), 40, "float32", False)
    got = _backward(gpu_lib, ids, dout, torch.empty((40, 24), device="cuda"), False, 1.0)
    assert torch.isfinite(got).all()


@pytest.mark.parametrize("T", [40, 3000, 20000])
def test_same_bits(gpu_lib, T):
    """Repeated calls, and a workspace for more tokens, give the same bits."""
    import torch
    say(f"case embed backward same bits T={T}")
    ids, dout, start = _ids(T, 50, spread="text"), _rnd(T, 100), _rnd(50, 100, seed=4)
    first = _backward(gpu_lib, ids, dout, start, True, 1.0).clone()
    for most in (T, T + 1, 4 * T):
        assert torch.equal(_backward(gpu_lib, ids, dout, start, True, 1.0, most), first)


@pytest.mark.parametrize("T", [100, 9000])
def test_graph_and_streams(gpu_lib, T):
    """Forward and backward captured together and replayed on new inputs between eager work; a stream of the caller's."""
    import torch
    tw, V, d = gpu_lib, 77, 20
    say(f"case embed graph T={T}")
    ids, table, out = _ids(T, V), _rnd(V, d), torch.empty((T, d), device="cuda")
    dtable, ws = torch.empty((V, d), device="cuda"), tw.embed_workspace(T, V, d)

    def step(stream=None):
        tw.twell_embed_forward(ids, table, out, scale=2.0, stream=stream)
        tw.twell_embed_backward(ids, out, dtable, ws, scale=0.5, stream=stream)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(4):
        ids.copy_(_ids(T, V, seed=k, spread=("uniform", "text", "one", "uniform")[k]))
        table.copy_(_rnd(V, d, seed=k + 9))
        out.fill_(float("nan"))
        dtable.fill_(float("nan"))
        graph.replay()
        got = out.clone(), dtable.clone()
        step()
        assert torch.equal(out, got[0]) and torch.equal(dtable, got[1])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        out.fill_(0)
        side.wait_stream(torch.cuda.current_stream())
        step(stream=side)
        side.synchronize()
        assert torch.equal(out, got[0]) and torch.equal(dtable, got[1])


def test_host_tensors_are_refused(gpu_lib):
    import torch
    say("case embed, host tensors")
    with pytest.raises(ValueError):
        gpu_lib.twell_embed_forward(_ids(3, 4), torch.zeros(4, 8), torch.zeros(3, 8))
    with pytest.raises(ValueError):
        gpu_lib.twell_embed_forward(torch.zeros(3, dtype=torch.int64), _rnd(4, 8), torch.zeros((3, 8), device="cuda"))
    with pytest.raises(ValueError):
        gpu_lib.twell_embed_backward(_ids(3, 4), _rnd(3, 8), _rnd(4, 8), torch.zeros(4096, dtype=torch.uint8))
