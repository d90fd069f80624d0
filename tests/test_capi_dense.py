"""The C ABI of the dense layer's operators on the host (no GPU needed): bad
arguments are rejected before anything is launched."""

import ctypes

import unstructured_sparse_transformer_amd as tw

GOOD = 4096  # an aligned, never dereferenced fake device address
NULL, ALIGN, SHAPE, UNSUPPORTED, WORKSPACE = -1, -2, -3, -4, -6


def _adamw(**kw):
    t = tw.TwellAdamWTensorT(n=1000, p=GOOD, grad=GOOD, m=GOOD, v=GOOD, pdtype=0, gdtype=1)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


def _step(t, count=1, bits=32, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, step=1, scale=None):
    return tw.load().twell_adamw_step(ctypes.byref(t) if t is not None else None, count, bits, lr, b1, b2, eps, step, 0,
                                      scale, None)


def test_adamw_validation():
    assert _step(None) == NULL
    assert _step(None, count=0) == 0
    assert _step(_adamw(n=0)) == 0
    assert _step(_adamw(), count=-1) == SHAPE
    assert _step(_adamw(n=-1)) == SHAPE
    for k in ("p", "grad", "m", "v"):
        assert _step(_adamw(**{k: None})) == NULL
    assert _step(_adamw(), bits=8) == NULL                              # no scales
    assert _step(_adamw(m_scale=GOOD, v_scale=GOOD + 2), bits=8) == ALIGN
    assert _step(_adamw(p=GOOD + 2)) == ALIGN
    assert _step(_adamw(grad=GOOD + 1)) == ALIGN
    assert _step(_adamw(copy=GOOD + 1)) == ALIGN
    assert _step(_adamw(), scale=GOOD + 2) == ALIGN
    assert _step(_adamw(), bits=16) == UNSUPPORTED
    assert _step(_adamw(pdtype=2)) == UNSUPPORTED
    assert _step(_adamw(gdtype=-1)) == UNSUPPORTED
    nan = float("nan")
    for kw in (dict(step=0), dict(b1=1.0), dict(b1=-0.1), dict(b2=1.0), dict(eps=0.0), dict(lr=-1.0), dict(lr=nan),
               dict(b1=nan), dict(b2=nan), dict(eps=nan)):
        assert _step(_adamw(), **kw) == SHAPE, kw
    lib = tw.load()
    assert lib.twell_adamw_unpack(None, 1, None) == NULL
    assert lib.twell_adamw_unpack(None, 0, None) == 0
    t = _adamw(m_scale=GOOD, v_scale=GOOD, m_values=GOOD)
    assert lib.twell_adamw_unpack(ctypes.byref(t), 1, None) == NULL      # v_values
    t.v_values = GOOD + 2
    assert lib.twell_adamw_unpack(ctypes.byref(t), 1, None) == ALIGN


def _bn(**kw):
    t = tw.TwellBlockNormT(T=8, d=64, kind=0, post=1, eps=1e-6, alpha=1.0, gate_span=0)
    for k, v in kw.items():
        setattr(t, k, v)
    return ctypes.byref(t)


def test_block_norm_validation():
    lib = tw.load()
    f = lib.twell_block_norm_forward
    assert f(None, GOOD, GOOD, GOOD, GOOD, None) == NULL
    assert f(_bn(T=0), None, None, None, None, None) == 0
    assert f(_bn(), None, GOOD, GOOD, GOOD, None) == NULL              # res
    assert f(_bn(), GOOD, GOOD, None, None, None) == NULL              # neither out nor n
    assert f(_bn(), GOOD, None, GOOD, None, None) == NULL              # out without a block is not written
    assert f(_bn(gate_span=2), GOOD, GOOD, GOOD, GOOD, None) == NULL   # gate
    assert f(_bn(), GOOD + 2, GOOD, GOOD, GOOD, None) == ALIGN
    assert f(_bn(w_pre=GOOD + 2), GOOD, GOOD, GOOD, GOOD, None) == ALIGN
    assert f(_bn(rdtype=1, ydtype=1, ndtype=1), GOOD, GOOD, GOOD + 1, GOOD, None) == ALIGN
    for kw in (dict(kind=2), dict(d=8193), dict(rdtype=2), dict(ydtype=-1), dict(ndtype=5), dict(wdtype=2)):
        assert f(_bn(**kw), GOOD, GOOD, GOOD, GOOD, None) == UNSUPPORTED, kw
    for kw in (dict(T=-1), dict(T=(1 << 30) + 1), dict(d=0), dict(gate_span=-1), dict(eps=0.0), dict(eps=float("nan"))):
        assert f(_bn(**kw), GOOD, GOOD, GOOD, GOOD, None) == SHAPE, kw
    size = lib.twell_block_norm_workspace_bytes
    assert size(-1, 64) == 0 and size(8, 0) == 0 and size(8, 8193) == 0 and size(0, 64) == 0
    need = size(8, 64)
    assert need > 0

    def b(bn=None, out=GOOD, y=GOOD, dout=GOOD, dn=GOOD, dndtype=0, dres=GOOD, dy=GOOD, dgate=None, dw=None, ws=GOOD,
          nbytes=need):
        return lib.twell_block_norm_backward(bn or _bn(), out, y, dout, dn, dndtype, dres, dy, dgate, dw, None, None, None,
                                             ws, nbytes, None)
    assert b(dout=None, dn=None) == NULL
    assert b(out=None) == NULL
    assert b(dres=None) == NULL
    assert b(dy=None) == NULL
    assert b(bn=_bn(gate_span=2, gate=GOOD)) == NULL                    # dgate
    assert b(dw=GOOD + 2) == ALIGN
    assert b(dndtype=3) == UNSUPPORTED
    assert b(ws=None) == WORKSPACE and b(nbytes=need - 1) == WORKSPACE and b(ws=GOOD + 128) == ALIGN


def test_glu_validation():
    lib = tw.load()

    def f(x=GOOD, wg=GOOD, wu=GOOD, T=8, d=64, F=128, vd=1, act=1, h=GOOD, g=None, u=None):
        return lib.twell_glu_forward(x, wg, wu, T, d, F, vd, act, h, g, u, None, 0, None)

    for k in ("x", "wg", "wu", "h"):
        assert f(**{k: None}) == NULL and f(**{k: GOOD + 8}) == ALIGN, k
    assert f(g=GOOD + 2) == ALIGN and f(u=GOOD + 8) == ALIGN
    assert f(T=0, x=None, h=None) == 0
    for kw in (dict(T=-1), dict(T=(1 << 30) + 1), dict(d=0), dict(d=96), dict(F=100), dict(F=0), dict(d=-64)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(vd=2), dict(act=-1), dict(act=4), dict(d=(1 << 20) + 64), dict(F=(1 << 19) + 64)):
        assert f(**kw) == UNSUPPORTED, kw
    assert f(T=(1 << 31) - 1, F=1 << 19) == SHAPE
    size = lib.twell_glu_backward_workspace_bytes
    assert size(8, 60, 128, 1) == 0 and size(-1, 64, 128, 1) == 0 and size(8, 64, 128, 3) == 0
    need = size(8, 64, 128, 1)
    assert need >= 64 * 256 * 2

    def b(x=GOOD, wg=GOOD, wu=GOOD, g=GOOD, u=GOOD, dh=GOOD, dx=GOOD, dwg=GOOD, dwu=GOOD, ws=GOOD, nbytes=need):
        return lib.twell_glu_backward(x, wg, wu, g, u, dh, 8, 64, 128, 1, 1, dx, dwg, dwu, ws, nbytes, None)

    for k in ("x", "wg", "wu", "g", "u", "dh"):
        assert b(**{k: None}) == NULL and b(**{k: GOOD + 4}) == ALIGN, k
    assert b(dx=None, dwg=None, dwu=None) == NULL and b(dwg=None) == NULL and b(dwu=None) == NULL
    for k in ("dx", "dwg", "dwu"):
        assert b(**{k: GOOD + 8}) == ALIGN, k
    assert b(ws=None) == WORKSPACE and b(nbytes=need - 1) == WORKSPACE and b(ws=GOOD + 16) == ALIGN
