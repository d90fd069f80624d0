"""What the layers of the training example keep: with the products in 8 bits a further layer has no buffer of T x F in 16
bits."""

import importlib.util
import os

import pytest

from helpers import say

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example(gpu_lib):
    spec = importlib.util.spec_from_file_location("train_layer", os.path.join(ROOT, "examples", "train_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_a_further_layer_s_memory(example):
    """Of a layer more (T = 2048, d = 64, F = 4096; the optimizer's states, the rows of d and the weights are the same):
    16 bits keep g, u and h, and have dh and the backward pass's workspace of 2 T F, 12 bytes an element of T x F; 8 bits
    keep 2 (1 + 2 / 32) bytes."""
    import torch
    T, d, F = 2048, 64, 4096

    def more(ffn):
        torch.cuda.synchronize()
        at = [torch.cuda.memory_allocated()]
        for layers in (1, 2, 3):
            stack = example.Stack(T, d, F, layers, ffn)  # noqa: F841 (alive while it is measured)
            at.append(torch.cuda.memory_allocated() - at[0])
            del stack
        assert at[3] - at[2] == at[2] - at[1]
        return at[3] - at[2]

    say("case train memory")
    wide, narrow = more(example.Gated), more(example.GatedKept8)
    saved = (12 - 2.125) * T * F
    assert wide - narrow > 0.99 * saved, f"{(wide - narrow) / (T * F):.3f} bytes an element"


def test_gradients_of_three_layers(example):
    """Shared buffers: the gradients are those of layers with buffers of their own."""
    import torch
    say("case train shared buffers")
    T, d, F = 130, 128, 512
    got = []
    for own in (False, True):
        stack = example.Stack(T, d, F, 3, example.GatedKept8)
        if own:
            for k in (1, 2):
                f = stack.ffn[k]
                f.h, f.dh = torch.empty_like(f.h), torch.empty_like(f.dh)
                f.ws = None if f.ws is None else torch.empty_like(f.ws)
                f.ws_backward = torch.empty_like(f.ws_backward)
        gen = torch.Generator(device="cuda").manual_seed(4)
        x, dn = (torch.randn((T, d), generator=gen, device="cuda") for _ in range(2))
        n = stack.forward(x).clone()
        dx = stack.backward(dn).clone()
        got.append([n, dx] + [g for f in stack.ffn for g in f.grads] + stack.dw_pre + stack.dw_post)
        assert all(torch.isfinite(t).all() for t in got[-1])
    assert all(torch.equal(a, b) for a, b in zip(*got))
