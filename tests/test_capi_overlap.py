"""Calls of the token operators and of the 8-bit activations whose result lies in part in what they read are refused on the
host (no GPU needed)."""

import ctypes

import pytest

import unstructured_sparse_transformer_amd as tw

AT = 1 << 30  # a never dereferenced fake device address
SHAPE = -3


def _places(size, other):
    """Offsets of `size` bytes against `other` bytes at which they share some: the same start, one element in, the last ones."""
    return [off for off in (0, 4, -4, (other - 1) // 4 * 4, 4 - size) if -size < off < other]


@pytest.mark.parametrize("T,V,d", [(8, 10, 16), (1, 1, 1), (5, 300, 1001)])
def test_embed_forward(T, V, d):
    lib = tw.load()
    table, out, ids = V * d * 2, T * d * 4, T * 8
    call = lambda i, t, o: lib.twell_embed_forward(i, 64, T, t, V, d, tw.TWELL_BF16, 1.0, o, tw.TWELL_F32, None)  # noqa: E731
    for off in _places(out, table):
        assert call(AT * 64, AT, AT + off) == SHAPE, off
    for off in _places(out, ids):
        assert call(AT, AT * 64, AT + off) == SHAPE, off


@pytest.mark.parametrize("add", [0, 1])
@pytest.mark.parametrize("T,V,d", [(8, 10, 16), (1, 1, 1), (5, 300, 1001)])
def test_embed_backward(T, V, d, add):
    lib = tw.load()
    dtable, dout, ids = V * d * 4, T * d * 4, T * 4
    n = lib.twell_embed_workspace_bytes(T, V, d)
    call = lambda i, g, o: lib.twell_embed_backward(i, 32, T, g, tw.TWELL_F32, V, d, 1.0, add, o, tw.TWELL_F32, AT * 128, n, None)  # noqa: E731
    for off in _places(dtable, dout):
        assert call(AT * 64, AT, AT + off) == SHAPE, off
    for off in _places(dtable, ids):
        assert call(AT, AT * 64, AT + off) == SHAPE, off


@pytest.mark.parametrize("T,d", [(8, 32), (1, 1), (5, 1001)])
@pytest.mark.parametrize("vd", [0, 1])
def test_act_pack(T, d, vd):
    lib = tw.load()
    es, scales = (4, 2)[vd], T * -(-d // 32) * 2
    pack = lambda x, c, s: lib.twell_act_pack(x, T, d, vd, ctypes.byref(tw.TwellPackedT(c, s)), None)  # noqa: E731
    unpack = lambda x, c, s: lib.twell_act_unpack(ctypes.byref(tw.TwellPackedT(c, s)), T, d, vd, x, None)  # noqa: E731
    for f in (pack, unpack):
        for off in _places(T * d, T * d * es):
            assert f(AT, AT + off, AT * 64) == SHAPE, off
        for off in _places(scales, T * d * es):
            assert f(AT, AT * 64, AT + off) == SHAPE, off


@pytest.mark.gpu
def test_side_by_side(gpu_lib):
    """Neighbours in one buffer share no byte and are served."""
    import torch
    T, V, d = 6, 9, 5
    buf = torch.zeros(2 * T * d + V * d, device="cuda")
    out, table, dout = buf[:T * d].view(T, d), buf[T * d:T * d + V * d].view(V, d), buf[T * d + V * d:].view(T, d)
    table.copy_(torch.arange(V * d, device="cuda").view(V, d))
    ids = torch.tensor([3, 0, 8, -1, 3, 3], device="cuda")
    tw.twell_embed_forward(ids, table, out, scale=2.0)
    want = table[ids] * 2
    want[3] = 0
    assert torch.equal(out, want)
    dout.fill_(1)
    tw.twell_embed_backward(ids, dout, table, tw.embed_workspace(T, V, d))
    assert table[:, 0].tolist() == [1, 0, 0, 3, 0, 0, 0, 0, 1] and torch.equal(out, want) and (dout == 1).all()
    with pytest.raises(tw.TwellError):
        tw.twell_embed_backward(ids, table[1:7], table, tw.embed_workspace(T, V, d))
    with pytest.raises(tw.TwellError):
        tw.twell_embed_forward(ids, table, table[:T])
    assert table[:, 0].tolist() == [1, 0, 0, 3, 0, 0, 0, 0, 1]
