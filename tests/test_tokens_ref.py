"""The 64-bit formulas of tokens_ref.py against differences and against torch's
own derivatives (CPU)."""

import math

import pytest
import torch

import tokens_ref


def _rnd(*shape, seed=1):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def _difference(f, x, h=1e-6):
    out = torch.zeros_like(x)
    for i in range(x.numel()):
        d = torch.zeros_like(x).view(-1)
        d[i] = h
        d = d.view_as(x)
        out.view(-1)[i] = (f(x + d) - f(x - d)) / (2 * h)
    return out


def test_embedding_gradient():
    ids, table, dout = torch.tensor([2, 0, 2, -1, 5, 1, 2]), _rnd(5, 3), _rnd(7, 3, seed=2)
    loss = lambda t: float((tokens_ref.embed_forward(ids, t, 0.5)[0] * dout).sum())  # noqa: E731
    got = tokens_ref.embed_backward(ids, dout, 5, 0.5)[0]
    assert torch.allclose(got, _difference(loss, table), atol=1e-8)
    assert (got[3:] == 0).all()
    assert torch.allclose(tokens_ref.embed_backward(ids, dout, 5, 0.5, table)[0], got + table)


@pytest.mark.parametrize("scale", [1.0, 0.7])
def test_log_probabilities(scale):
    z, targets = _rnd(6, 9) * 3, torch.tensor([0, 8, 3, -1, 9, 4])
    z[1, 2:5] = -math.inf
    z[5] = -math.inf
    got, idx = tokens_ref.logprob_forward(z, targets, scale, k=4)
    want = torch.log_softmax(z[:5] * scale, 1)
    at = targets[:3]
    assert torch.allclose(got["logp"][0][:3], want[:3].gather(1, at[:, None])[:, 0], atol=1e-12)
    assert got["logp"][0][3:5].tolist() == [0, 0] and got["logp"][0][5] == -math.inf
    H = torch.distributions.Categorical(logits=z[[0, 2, 3, 4]] * scale).entropy()
    assert torch.allclose(got["entropy"][0][[0, 2, 3, 4]], H, atol=1e-12)
    assert got["entropy"][0][5] == 0 and got["norm"][0][5].tolist() == [-math.inf, 0]
    assert torch.allclose(got["norm"][0][:5, 0] * scale + got["norm"][0][:5, 1], torch.logsumexp(z[:5] * scale, 1))
    assert torch.equal(idx[5], torch.arange(4)) and torch.equal(idx[0], torch.topk(z[0], 4).indices)


@pytest.mark.parametrize("scale", [1.0, 0.7])
def test_log_probabilities_gradient(scale):
    z, targets = _rnd(4, 7) * 2, torch.tensor([0, 6, -1, 3])
    dlogp, dent = _rnd(4, seed=5), _rnd(4, seed=6)

    def loss(z):
        got, _ = tokens_ref.logprob_forward(z, targets, scale)
        return float((got["logp"][0] * dlogp).sum() + (got["entropy"][0] * dent).sum())

    got, _ = tokens_ref.logprob_forward(z, targets, scale)
    back = lambda d, h: tokens_ref.logprob_backward(z, targets, got["norm"][0], d, scale, got["entropy"][0], h)[0]  # noqa: E731
    assert torch.allclose(back(dlogp, dent), _difference(loss, z), atol=1e-7)
    assert torch.allclose(back(dlogp, None) + back(None, dent), back(dlogp, dent), atol=1e-12)
    z[0, 3] = z[1] = -math.inf
    got, _ = tokens_ref.logprob_forward(z, targets, scale)
    dz = tokens_ref.logprob_backward(z, targets, got["norm"][0], dlogp, scale, got["entropy"][0], dent)[0]
    assert dz[0, 3] == 0 and (dz[1] == 0).all() and torch.isfinite(dz).all()


def test_pack():
    x = torch.randn((5, 70), generator=torch.Generator().manual_seed(3))
    x[1, 32:64] = 0
    x[2, 5] = math.nan
    x[3, 69] = -math.inf
    x[4] *= 1e-33
    code, scale, value = tokens_ref.pack(x)
    assert code.shape == (5, 70) and scale.shape == (5, 3)
    assert torch.equal(scale[torch.isfinite(scale)], scale[torch.isfinite(scale)].bfloat16().float())
    assert torch.isnan(value[2, :32]).all() and torch.isfinite(value[2, 32:]).all()
    assert torch.isnan(value[3, 64:]).all() and torch.isfinite(value[3, :64]).all()
    assert (value[1, 32:64] == 0).all() and (value[4] == 0).all()
    fine = torch.isfinite(value)
    fine[4] = False
    off = (value.double() - x.double()).abs()
    assert (off <= tokens_ref.kept_bound(x.double().nan_to_num(0, 0, 0), 0.0))[fine].all()
    assert int(code[0].abs().max()) in (126, 127)
