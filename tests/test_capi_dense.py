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
