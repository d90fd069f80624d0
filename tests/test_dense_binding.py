"""The Python side of the dense layer's operators on the host (no GPU needed):
what a call hands to the C side."""

import ctypes

import pytest
import torch

import unstructured_sparse_transformer_amd as tw

CPU = -1  # a host tensor's device number, in the place of a GPU's


@pytest.mark.parametrize("span", [7, 8, (1 << 31) - 1, 1 << 31, 1 << 32, (1 << 32) + 1, (1 << 32) + 3, 1 << 40])
def test_gate_row_of_any_span(span):
    """One gate row for all rows is that, however large the span is that says so."""
    rows, gate = torch.zeros(7, 16), torch.zeros(1, 16)
    o = tw.BlockNorm().desc("f", CPU, rows, rows, gate, span)
    assert o.T == 7 and o.gate_span >= 7


def test_counts_past_32_bits_are_refused():
    """More rows than an argument holds stay more than the C side takes."""
    T, most = (1 << 32) + 128, 1 << 30
    rows = torch.zeros((T, 0))
    assert tw.BlockNorm().desc("f", CPU, rows, None, None, 0).T > most
    with pytest.raises(tw.TwellError):
        tw._check("f", tw.load().twell_block_norm_forward(tw.BlockNorm().desc("f", CPU, rows, None, None, 0), None, None,
                                                          None, None, None))
    for dt in (torch.bfloat16, torch.float32):
        assert tw.twell_glu_workspace_bytes(128, 4096, 512, dt) > 0
        assert tw.twell_glu_workspace_bytes(T, 4096, 512, dt) == 0
        assert tw.twell_glu_workspace_bytes(128, (1 << 32) + 4096, 512, dt) == 0
        assert tw.twell_glu_backward_workspace_bytes(T, 128, 128, dt) == 0
        assert tw.twell_glu_backward_workspace_bytes(128, 128, (1 << 32) + 128, dt) == 0
    assert tw.twell_block_norm_workspace_bytes(T, 64) == 0
    assert tw.twell_block_norm_workspace_bytes(64, (1 << 32) + 64) == 0


def test_adamw_eps_is_one_of_32_bits():
    """An eps that is 0 as a float divides 0 by 0 where an element has no moments yet: refused as 0 is."""
    at = 4096  # an aligned, never dereferenced fake device address
    t = tw.TwellAdamWTensorT(n=1000, p=at, grad=at, m=at, v=at)
    step = lambda eps: tw.load().twell_adamw_step(  # noqa: E731
        ctypes.byref(t), 1, 32, 1e-3, 0.9, 0.99, eps, 1, 0, None, None)
    assert [step(eps) for eps in (0.0, 1e-46, 7e-46, 5e-324, float("nan"))] == [-3] * 5


def test_a_block_s_tensors_need_the_block(monkeypatch):
    """A gate, or a place for a block's gradient, without the block's y is refused, not left as it is."""
    monkeypatch.setattr(tw, "_device", lambda fn, t: CPU)
    rows, gate, bn = torch.ones(6, 16), torch.ones(2, 16), tw.BlockNorm()
    new = lambda: torch.empty(6, 16)  # noqa: E731
    with pytest.raises(ValueError, match="gate"):
        tw.twell_block_norm_forward(bn, rows, None, None, new(), gate=gate, gate_span=3, stream=0)
    back = lambda dy, **kw: tw.twell_block_norm_backward(bn, rows, None, rows, rows, new(), dy, None, stream=0, **kw)  # noqa: E731
    with pytest.raises(ValueError, match="gate"):
        back(None, gate=gate, gate_span=3, dgate=gate.clone())
    with pytest.raises(ValueError, match="dy"):
        back(new())


def test_weights_that_moved(monkeypatch):
    """A weight whose data is another tensor's by the time of a call is read where it is then, and checked anew."""
    monkeypatch.setattr(tw, "_device", lambda fn, t: CPU)
    rows, w, b = torch.ones(6, 16), torch.ones(16), torch.zeros(16)
    bn = tw.BlockNorm(w_pre=w, b_pre=b)
    desc = lambda: bn.desc("f", CPU, rows, None, None, 0)  # noqa: E731
    assert (desc().w_pre, desc().b_pre, desc().wdtype) == (w.data_ptr(), b.data_ptr(), tw.TWELL_F32)
    old = w.data
    w.data = torch.ones(16)
    assert old.data_ptr() != w.data_ptr()
    assert (desc().w_pre, desc().b_pre) == (w.data_ptr(), b.data_ptr())
    w.data, b.data = w.data.bfloat16(), b.data.bfloat16()
    assert (desc().w_pre, desc().wdtype) == (w.data_ptr(), tw.TWELL_BF16)
    good, at = b.data, b.data_ptr()
    for bad in (torch.zeros(8, dtype=torch.bfloat16), torch.zeros(16), torch.zeros(32, dtype=torch.bfloat16)[::2]):
        b.data = bad
        with pytest.raises((ValueError, TypeError)):
            desc()
    b.data = good
    assert (desc().w_pre, desc().b_pre) == (w.data_ptr(), at)
