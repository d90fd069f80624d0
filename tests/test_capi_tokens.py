"""The C ABI of the token operators and the 8-bit activations on the host (no GPU
needed): bad arguments are rejected before anything is launched."""

import ctypes

import pytest

import unstructured_sparse_transformer_amd as tw

GOOD = 4096  # an aligned, never dereferenced fake device address
NULL, ALIGN, SHAPE, UNSUPPORTED, WORKSPACE = -1, -2, -3, -4, -6
NAN, INF = float("nan"), float("inf")
BIG = 1 << 30


def test_embed_forward():
    def f(ids=GOOD, bits=64, T=8, table=GOOD, V=10, d=16, vd=1, scale=1.0, out=GOOD, od=0):
        return tw.load().twell_embed_forward(ids, bits, T, table, V, d, vd, scale, out, od, None)

    assert f(ids=None) == NULL and f(table=None) == NULL and f(out=None) == NULL
    assert f(T=0, ids=None, out=None) == 0
    assert f(ids=GOOD + 4) == ALIGN and f(bits=32, ids=GOOD + 2) == ALIGN
    assert f(table=GOOD + 1) == ALIGN and f(out=GOOD + 2) == ALIGN
    for kw in (dict(bits=16), dict(bits=0), dict(vd=2), dict(od=-1)):
        assert f(**kw) == UNSUPPORTED, kw
    for kw in (dict(T=-1), dict(T=BIG + 1), dict(V=0), dict(V=BIG + 1), dict(d=0), dict(d=(1 << 20) + 1),
               dict(T=BIG, d=1 << 20)):
        assert f(**kw) == SHAPE, kw


def test_embed_backward():
    size = tw.load().twell_embed_workspace_bytes
    assert size(-1, 10, 16) == 0 and size(8, 0, 16) == 0 and size(8, 10, 0) == 0 and size(BIG, 10, 1 << 20) == 0
    need = size(8, 10, 16)
    assert need > 0

    def f(ids=GOOD, bits=64, T=8, dout=GOOD, dd=1, V=10, d=16, scale=1.0, add=0, dtable=GOOD, vd=0, ws=GOOD, n=need):
        return tw.load().twell_embed_backward(ids, bits, T, dout, dd, V, d, scale, add, dtable, vd, ws, n, None)

    assert f(ids=None) == NULL and f(dout=None) == NULL and f(dtable=None) == NULL
    assert f(ids=GOOD + 4) == ALIGN and f(dout=GOOD + 1) == ALIGN and f(dtable=GOOD + 2) == ALIGN
    assert f(T=0, ids=None, dout=None, add=1, ws=None, n=0) == 0
    assert f(ws=None) == WORKSPACE and f(n=need - 1) == WORKSPACE and f(ws=GOOD + 128) == ALIGN
    for kw in (dict(bits=8), dict(vd=2), dict(dd=3)):
        assert f(**kw) == UNSUPPORTED, kw
    for kw in (dict(T=-1), dict(T=BIG + 1), dict(V=0), dict(d=0), dict(d=(1 << 20) + 1)):
        assert f(**kw) == SHAPE, kw


def test_logprob_forward():
    size = tw.load().twell_logprob_workspace_bytes
    assert size(-1, 10, 0) == 0 and size(8, 0, 0) == 0 and size(8, 10, 11) == 0 and size(8, 100, 65) == 0
    need = size(8, 100000, 5)
    assert need > 0 and size(8, 64, 5) == 0 and size(1 << 20, 100000, 5) >= need

    def f(z=GOOD, ld=100000, T=8, V=100000, vd=1, scale=1.0, t=GOOD, bits=64, logp=GOOD, norm=GOOD, ent=GOOD, tl=GOOD,
          ti=GOOD, k=5, ws=GOOD, n=need):
        return tw.load().twell_logprob_forward(z, ld, T, V, vd, scale, t, bits, logp, norm, ent, tl, ti, k, ws, n, None)

    assert f(z=None) == NULL and f(t=None) == NULL and f(tl=None) == NULL and f(ti=None) == NULL
    assert f(logp=None, norm=None, ent=None, k=0) == NULL
    assert f(T=0, z=None) == 0
    for kw in (dict(z=GOOD + 1), dict(t=GOOD + 4), dict(logp=GOOD + 2), dict(norm=GOOD + 1), dict(ent=GOOD + 2),
               dict(tl=GOOD + 2), dict(ti=GOOD + 1), dict(ws=GOOD + 16), dict(vd=0, z=GOOD + 2)):
        assert f(**kw) == ALIGN, kw
    for kw in (dict(vd=2), dict(bits=63), dict(k=65)):
        assert f(**kw) == UNSUPPORTED, kw
    for kw in (dict(T=-1), dict(T=BIG + 1), dict(V=0, ld=0), dict(V=BIG + 1, ld=BIG + 1), dict(ld=99999), dict(ld=(1 << 40) + 1),
               dict(k=-1), dict(V=4, k=5), dict(scale=0.0), dict(scale=-1.0), dict(scale=NAN), dict(scale=INF),
               dict(T=BIG, V=BIG, ld=BIG)):
        assert f(**kw) == SHAPE, kw
    assert f(ws=None) == WORKSPACE and f(n=64) == WORKSPACE


def test_logprob_backward():
    def f(z=GOOD, ld=100, T=8, V=100, vd=1, scale=1.0, t=GOOD, bits=64, norm=GOOD, ent=GOOD, dl=GOOD, de=GOOD, dz=GOOD, ldd=100):
        return tw.load().twell_logprob_backward(z, ld, T, V, vd, scale, t, bits, norm, ent, dl, de, dz, ldd, None)

    assert f(T=0, z=None, dz=None) == 0
    for kw in (dict(z=None), dict(dz=None), dict(norm=None), dict(t=None), dict(ent=None), dict(dl=None, de=None)):
        assert f(**kw) == NULL, kw
    for kw in (dict(z=GOOD + 1), dict(dz=GOOD + 1), dict(norm=GOOD + 2), dict(t=GOOD + 4), dict(ent=GOOD + 2), dict(dl=GOOD + 1),
               dict(de=GOOD + 3)):
        assert f(**kw) == ALIGN, kw
    for kw in (dict(vd=5), dict(bits=0)):
        assert f(**kw) == UNSUPPORTED, kw
    for kw in (dict(T=-1), dict(V=0), dict(ld=99), dict(ldd=99), dict(scale=0.0), dict(scale=NAN), dict(ldd=101)):
        assert f(**kw) == SHAPE, kw
    # dlogits partly in the logits' place: 8 rows of 100 bf16, 200 bytes apart
    for at in (2, 198, 200, 1598, -2, -200, -1598):
        assert f(dz=GOOD + at) == SHAPE, at
    for at, ld in ((198, 199), (300, 200), (1450, 400)):  # in the gaps of wider rows, but not all of a row
        assert f(dz=GOOD + at, ld=ld, ldd=ld) == SHAPE, (at, ld)
    assert f(dz=GOOD + 200, ld=200, ldd=300) == SHAPE


@pytest.mark.parametrize("rows", [1, 2, 7])
def test_logprob_backward_overlaps(rows):
    """Against the elements themselves: dlogits shares none with the logits, or lies in their place."""
    lib, V, es = tw.load(), 6, 4
    for ld in (6, 7, 12, 13, 20):
        for ldd in (6, 7, 12, 13, 20):
            a = {t * ld + v for t in range(rows) for v in range(V)}
            for off in range(-rows * 21, rows * 21):
                b = {off + t * ldd + v for t in range(rows) for v in range(V)}
                # (a NULL norm ends the calls that are not refused for their places)
                got = lib.twell_logprob_backward(GOOD * 16, ld, rows, V, 0, 1.0, GOOD, 64, GOOD, None, GOOD + 1, None,
                                                 GOOD * 16 + off * es, ldd, None)
                assert got in (SHAPE, ALIGN)
                if got == ALIGN:
                    assert not a & b or (off == 0 and (ld == ldd or rows == 1)), (ld, ldd, off)
                elif ld == ldd:
                    assert a & b, (ld, off)


def _pk(code=GOOD, scale=GOOD):
    return ctypes.byref(tw.TwellPackedT(code, scale))


def test_act_pack():
    lib = tw.load()
    for f in (lambda x=GOOD, T=8, d=16, vd=1, p=_pk(): lib.twell_act_pack(x, T, d, vd, p, None),
              lambda x=GOOD, T=8, d=16, vd=1, p=_pk(): lib.twell_act_unpack(p, T, d, vd, x, None)):
        assert f(x=None) == NULL and f(p=None) == NULL and f(p=_pk(code=None)) == NULL and f(p=_pk(scale=None)) == NULL
        assert f(T=0, x=None, p=None) == 0
        assert f(x=GOOD + 1) == ALIGN and f(vd=0, x=GOOD + 2) == ALIGN and f(p=_pk(scale=GOOD + 1)) == ALIGN
        assert f(vd=2) == UNSUPPORTED
        for kw in (dict(T=-1), dict(T=BIG + 1), dict(d=0), dict(d=(1 << 20) + 1)):
            assert f(**kw) == SHAPE, kw


def test_threads_of_a_launch():
    """Sizes whose threads pass what a launch counts in 32 bits are refused on the host."""
    lib = tw.load()
    for T, d in ((BIG, 64), (BIG, 61), (1 << 24, 1 << 12)):
        assert lib.twell_embed_forward(GOOD, 64, T, GOOD, 10, d, 1, 1.0, GOOD, 1, None) == SHAPE, (T, d)
        assert lib.twell_embed_workspace_bytes(T, 10, d) == 0, (T, d)
    for T, d, vd in ((BIG, 1, 0), (BIG, 33, 1), (1 << 20, 1 << 15, 0), (1 << 20, 1 << 16, 1)):
        assert lib.twell_act_pack(GOOD, T, d, vd, _pk(), None) == SHAPE, (T, d, vd)
        assert lib.twell_act_unpack(_pk(), T, d, vd, GOOD, None) == SHAPE, (T, d, vd)


def test_glu_packed():
    lib = tw.load()
    size = lib.twell_glu_packed_workspace_bytes
    assert size(8, 60, 128) == 0 and size(-1, 64, 128) == 0
    big = size(128, 4096, 64)
    assert big > 0

    def f(x=GOOD, wg=GOOD, wu=GOOD, T=128, d=4096, F=64, act=1, h=GOOD, g=_pk(), u=_pk(), ws=GOOD, n=big):
        return lib.twell_glu_forward_packed(x, wg, wu, T, d, F, act, h, g, u, 1, ws, n, None)

    for k in ("x", "wg", "wu", "h"):
        assert f(**{k: None}) == NULL and f(**{k: GOOD + 8}) == ALIGN, k
    for k in ("g", "u"):
        assert f(**{k: None}) == NULL and f(**{k: _pk(code=None)}) == NULL and f(**{k: _pk(scale=None)}) == NULL
        assert f(**{k: _pk(code=GOOD + 8)}) == ALIGN and f(**{k: _pk(scale=GOOD + 1)}) == ALIGN
    assert f(T=0, x=None, g=None) == 0
    assert f(ws=None) == WORKSPACE and f(n=64) == WORKSPACE and f(ws=GOOD + 16) == ALIGN
    for kw in (dict(T=-1), dict(d=96), dict(F=100)):
        assert f(**kw) == SHAPE, kw
    assert f(act=4) == UNSUPPORTED
    need = lib.twell_glu_backward_workspace_bytes(8, 64, 128, 1)

    def b(x=GOOD, wg=GOOD, wu=GOOD, g=_pk(), u=_pk(), dh=GOOD, h=None, dx=GOOD, dwg=GOOD, dwu=GOOD, ws=GOOD, n=need):
        return lib.twell_glu_backward_packed(x, wg, wu, g, u, dh, 8, 64, 128, 1, h, dx, dwg, dwu, ws, n, None)

    for k in ("x", "wg", "wu", "dh"):
        assert b(**{k: None}) == NULL and b(**{k: GOOD + 4}) == ALIGN, k
    for k in ("g", "u"):
        assert b(**{k: None}) == NULL and b(**{k: _pk(code=GOOD + 8)}) == ALIGN and b(**{k: _pk(scale=None)}) == NULL
    assert b(dx=None, dwg=None, dwu=None) == NULL and b(dwg=None) == NULL and b(dwu=None) == NULL
    for k in ("dx", "dwg", "dwu", "h"):
        assert b(**{k: GOOD + 8}) == ALIGN, k
    assert b(ws=None) == WORKSPACE and b(n=need - 1) == WORKSPACE and b(ws=GOOD + 16) == ALIGN


ROWS = sorted({m + i for m in [32 * k for k in range(1, 41)] + [1 << k for k in range(11, 21)] for i in (-1, 0, 1)} |
              set(range(1, 300)) | set(range(301, 20000, 97)))


def _grows(size, label):
    last = 0
    for T in ROWS:
        n = size(T)
        assert n >= last, f"{label} T={T}: {n} bytes, {last} for fewer rows"
        last = n


@pytest.mark.parametrize("V,d", [(1, 1), (300, 3), (50001, 1001), (131072, 2048), (BIG, 4)])
def test_embed_workspace_takes_the_largest(V, d):
    """A workspace that is large enough but starts 16 bytes too late is refused for its alignment, one byte less than a
    call's own rows need for its size."""
    lib = tw.load()
    _grows(lambda T: lib.twell_embed_workspace_bytes(T, V, d), (V, d))
    n = lib.twell_embed_workspace_bytes(20000, V, d)
    call = lambda T, n: lib.twell_embed_backward(GOOD, 32, T, GOOD, 1, V, d, 1.0, 1, GOOD, 0, GOOD + 16, n, None)  # noqa: E731
    for T in ROWS:
        assert T > 20000 or call(T, n) == ALIGN, T
        assert call(T, lib.twell_embed_workspace_bytes(T, V, d) - 1) == WORKSPACE, T


@pytest.mark.parametrize("V", [24577, 50001, 131072, 262144, 1 << 24])
@pytest.mark.parametrize("k", [0, 1, 20, 64])
def test_logprob_workspace_takes_the_largest(V, k):
    lib = tw.load()
    assert lib.twell_logprob_workspace_bytes(1, 12288, k) == 0  # rows that are never cut
    _grows(lambda T: lib.twell_logprob_workspace_bytes(T, V, k) if T <= 20000 else 1 << 60, (V, k))
    for most in (1, 7, 64, 777, 1024, 20000):
        n = lib.twell_logprob_workspace_bytes(most, V, k)
        for T in ROWS:
            if T <= min(most, 500):
                got = lib.twell_logprob_forward(GOOD, V, T, V, 1, 1.0, GOOD, 64, GOOD, GOOD, GOOD, GOOD, GOOD, k, GOOD + 16, n,
                                                None)
                assert got == ALIGN, (most, T, got)


def test_counts_past_32_bits_are_refused():
    wide = (1 << 32) + 64
    assert tw.twell_embed_workspace_bytes(64, 100, 64) > 0
    for sizes in ((wide, 100, 64), (64, wide, 64), (64, 100, wide)):
        assert tw.twell_embed_workspace_bytes(*sizes) == 0
    assert tw.twell_logprob_workspace_bytes(64, 100000, 5) > 0
    for sizes in ((wide, 100000, 5), (64, wide, 5), (64, 100000, 1 << 32)):
        assert tw.twell_logprob_workspace_bytes(*sizes) == 0
    assert tw.twell_glu_packed_workspace_bytes(128, 4096, 64) > 0
    for sizes in ((wide, 4096, 64), (128, wide, 64), (128, 4096, wide)):
        assert tw.twell_glu_packed_workspace_bytes(*sizes) == 0
