"""The Python side of the token operators and the 8-bit activations on the host (no
GPU needed): calls that are refused before the C side sees them."""

import pytest
import torch

import unstructured_sparse_transformer_amd as tw

CPU = -1  # a host tensor's device number, in the place of a GPU's


@pytest.fixture
def host(monkeypatch):
    """Host tensors pass for the current GPU's; a call that gets past the checks of its arguments ends in the C side."""
    monkeypatch.setattr(tw, "_device", lambda fn, t: CPU)


def _refused(call, *kinds, **changes):
    with pytest.raises(kinds or (ValueError, TypeError)):
        call(**changes)


def test_embed(host):
    ids, table, out, ws = torch.zeros(6, dtype=torch.int64), torch.zeros(9, 4), torch.zeros(6, 4), torch.zeros(512, dtype=torch.uint8)

    def f(ids=ids, table=table, out=out):
        tw.twell_embed_forward(ids, table, out, stream=0)

    def b(ids=ids, dout=out, dtable=table, ws=ws):
        tw.twell_embed_backward(ids, dout, dtable, ws, stream=0)

    for call in (f, b):
        _refused(call, TypeError, ids=ids.short())
        _refused(call, TypeError, ids=ids.float())
        _refused(call, ValueError, ids=torch.zeros((6, 1), dtype=torch.int64))
        _refused(call, ValueError, ids=torch.zeros(12, dtype=torch.int64)[::2])
    _refused(f, ValueError, out=torch.zeros(5, 4))
    _refused(f, ValueError, out=torch.zeros(4, 6).t())
    _refused(f, TypeError, out=out.half())
    _refused(f, TypeError, table=table.double())
    _refused(b, ValueError, dout=torch.zeros(6, 3))
    _refused(b, ValueError, dtable=torch.zeros(9, 8)[:, ::2])
    _refused(b, TypeError, dout=out.half())
    _refused(b, tw.TwellError, ws=None)
    _refused(b, tw.TwellError, ws=ws[:64])
    _refused(b, ValueError, ws=ws[::2])


def test_logprob(host):
    T, V, k = 3, 8, 2
    z, ids = torch.zeros(T, V), torch.zeros(T, dtype=torch.int32)
    v, norm = torch.zeros(T), torch.zeros(T, 2)
    top, idx = torch.zeros(T, k), torch.zeros((T, k), dtype=torch.int32)

    def f(logits=z, targets=ids, logp=v, norm=norm, scale=1.0, entropy=v, top_logp=top, top_idx=idx):
        tw.twell_logprob_forward(logits, targets, logp, norm, None, scale, entropy, top_logp, top_idx, stream=0)

    _refused(f, ValueError, targets=None)
    _refused(f, ValueError, logp=None)
    _refused(f, ValueError, top_idx=None)
    _refused(f, ValueError, top_logp=None)
    _refused(f, ValueError, norm=v)
    _refused(f, ValueError, entropy=torch.zeros(T + 1))
    _refused(f, TypeError, entropy=v.double())
    _refused(f, TypeError, top_idx=idx.long())
    _refused(f, ValueError, top_logp=torch.zeros(T, k + 1))
    _refused(f, TypeError, targets=ids.float())
    _refused(f, ValueError, targets=torch.zeros(T + 1, dtype=torch.int32))
    _refused(f, TypeError, logits=z.half())
    _refused(f, ValueError, logits=torch.zeros(V, T).t())
    _refused(f, ValueError, logits=torch.zeros(V).expand(T, V))
    _refused(f, ValueError, logits=torch.zeros(T, 2 * V)[:, ::2])
    _refused(f, tw.TwellError, scale=0.0)
    _refused(f, tw.TwellError, scale=float("nan"))
    _refused(f, tw.TwellError, top_idx=torch.zeros((T, 9), dtype=torch.int32), top_logp=torch.zeros(T, 9))  # k > V

    def b(logits=z, targets=ids, norm=norm, dlogp=v, dlogits=z, entropy=v, dentropy=v):
        tw.twell_logprob_backward(logits, targets, norm, dlogp, dlogits, 1.0, entropy, dentropy, stream=0)

    _refused(b, ValueError, targets=None)
    _refused(b, ValueError, entropy=None)
    _refused(b, tw.TwellError, dlogp=None, dentropy=None)
    _refused(b, ValueError, dlogits=torch.zeros(T, V + 1))
    _refused(b, ValueError, dlogits=z.bfloat16())
    _refused(b, ValueError, dlogits=torch.zeros(V, T).t())
    _refused(b, ValueError, dlogp=torch.zeros(T, 1))
    _refused(b, TypeError, dlogp=v.double())
    _refused(b, ValueError, norm=torch.zeros(2, T))


def test_act(host):
    x, p = torch.zeros(4, 64, dtype=torch.bfloat16), tw.PackedAct.empty(4, 64, device="cpu")
    assert p.scale.shape == (4, 2) and tw.PackedAct.empty(3, 33, device="cpu").scale.shape == (3, 2)
    for f in (lambda x=x, p=p: tw.twell_act_pack(x, p, stream=0), lambda x=x, p=p: tw.twell_act_unpack(p, x, stream=0)):
        _refused(f, TypeError, p=x)
        _refused(f, TypeError, x=x.half())
        _refused(f, ValueError, x=torch.zeros(64, 4).t())
        _refused(f, ValueError, p=tw.PackedAct.empty(4, 32, device="cpu"))
        _refused(f, TypeError, p=tw.PackedAct(p.code.to(torch.uint8), p.scale))
        _refused(f, TypeError, p=tw.PackedAct(p.code, p.scale.float()))
        _refused(f, ValueError, p=tw.PackedAct(p.code, p.scale[:, :1]))


def test_glu_packed(host):
    T, d, F = 4, 64, 128
    new = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    x, w, h, p = new(T, d), new(F, d), new(T, F), tw.PackedAct.empty(T, F, device="cpu")

    def f(x=x, wg=w, wu=w, act="silu", h=h, g=p, u=p):
        tw.twell_glu_forward_packed(x, wg, wu, act, h, g, u, stream=0)

    def b(x=x, wg=w, wu=w, act="silu", dh=h, g=p, u=p, dx=x, dwg=w, dwu=w, h=None):
        tw.twell_glu_backward_packed(x, wg, wu, g, u, dh, act, dx, dwg, dwu, None, h=h, stream=0)

    for call in (f, b):
        _refused(call, TypeError, x=x.float())
        _refused(call, TypeError, wu=w.float())
        _refused(call, ValueError, wg=w.t().contiguous())
        _refused(call, ValueError, act="tanh")
        _refused(call, TypeError, g=h)
        _refused(call, ValueError, u=tw.PackedAct.empty(T, F + 32, device="cpu"))
    _refused(f, TypeError, h=h.float())
    _refused(b, TypeError, dh=h.float())
    _refused(b, ValueError, h=new(T, d))
    _refused(b, tw.TwellError, dx=None, dwg=None, dwu=None)
    _refused(b, tw.TwellError, dwg=None)
    _refused(b, tw.TwellError)  # no workspace


def test_another_device_is_refused():
    """Without a GPU every tensor is on another device than the current GPU."""
    if torch.cuda.is_available():
        pytest.skip("host tensors meet a GPU here: the GPU tests have this case")
    for call in (lambda: tw.twell_act_pack(torch.zeros(2, 32), tw.PackedAct.empty(2, 32, device="cpu")),
                 lambda: tw.twell_embed_forward(torch.zeros(2, dtype=torch.int64), torch.zeros(3, 4), torch.zeros(2, 4)),
                 lambda: tw.twell_logprob_forward(torch.zeros(2, 3), None, None, torch.zeros(2, 2))):
        with pytest.raises((ValueError, RuntimeError)):
            call()
