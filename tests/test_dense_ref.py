"""The 64-bit formulas of dense_ref.py against differences and against torch's
own derivatives (CPU)."""

import pytest
import torch

import dense_ref


def _difference(f, x, h=1e-6):
    out = torch.zeros_like(x)
    for i in range(x.numel()):
        d = torch.zeros_like(x).view(-1)
        d[i] = h
        d = d.view_as(x)
        out.view(-1)[i] = (f(x + d) - f(x - d)) / (2 * h)
    return out


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("post", [True, False])
def test_norm_backward_against_differences(kind, post):
    gen = torch.Generator().manual_seed(4)
    rnd = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    T, d, span = 5, 6, 2
    val = dict(res=rnd(T, d), y=rnd(T, d), gate=rnd(3, d), w_post=rnd(d), b_post=rnd(d), w_pre=rnd(d), b_pre=rnd(d))
    dout, dn = rnd(T, d), rnd(T, d)

    def loss(**k):
        a = dict(val, **k)
        got = dense_ref.norm_forward(a["res"], a["y"], a["gate"], span, kind, 1e-3, 0.7, post,
                                     (a["w_post"], a["b_post"]), (a["w_pre"], a["b_pre"]))
        return float((got["out"][0] * dout).sum() + (got["n"][0] * dn).sum())

    out = dense_ref.norm_forward(val["res"], val["y"], val["gate"], span, kind, 1e-3, 0.7, post,
                                 (val["w_post"], val["b_post"]), (val["w_pre"], val["b_pre"]))["out"][0]
    got = dense_ref.norm_backward(out, val["y"], val["gate"], span, dout, dn, kind, 1e-3, 0.7, post,
                                  (val["w_post"], val["b_post"]), (val["w_pre"], val["b_pre"]))
    for k in val if post else ("res", "y", "gate", "w_pre", "b_pre"):
        want = _difference(lambda x: loss(**{k: x}), val[k])
        assert torch.allclose(got["d" + k][0], want, rtol=1e-6, atol=1e-6), k


@pytest.mark.parametrize("name", ["relu", "silu", "gelu", "gelu_tanh"])
def test_act(name):
    g = torch.linspace(-6, 6, 241, dtype=torch.float64) + 1e-3
    h = 1e-6
    diff = (dense_ref.act(g + h, name) - dense_ref.act(g - h, name)) / (2 * h)
    assert torch.allclose(dense_ref.act_grad(g, name), diff, atol=1e-8)
    theirs = {"relu": torch.relu, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
              "gelu_tanh": lambda x: torch.nn.functional.gelu(x, approximate="tanh")}[name](g)
    assert torch.allclose(dense_ref.act(g, name), theirs, atol=1e-12)


@pytest.mark.parametrize("name", ["relu", "silu", "gelu", "gelu_tanh"])
def test_glu_backward_against_differences(name):
    gen = torch.Generator().manual_seed(8)
    rnd = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    val = dict(x=rnd(3, 4), wg=rnd(5, 4), wu=rnd(5, 4))
    dh = rnd(3, 5)
    fwd = dense_ref.glu_forward(**val, name=name)
    got = dense_ref.glu_backward(val["x"], val["wg"], val["wu"], fwd["g"][0], fwd["u"][0], dh, name, torch.float32)
    for k in val:
        want = _difference(lambda x: float((dense_ref.glu_forward(**dict(val, **{k: x}), name=name)["h"][0] * dh).sum()),
                           val[k])
        assert torch.allclose(got["d" + k][0], want, rtol=1e-6, atol=1e-7), k
