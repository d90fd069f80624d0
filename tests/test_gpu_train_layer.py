"""The training example: its gradients against torch's derivatives of the same
layers in 64 bits, its optimizer step, and that it learns."""

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


def _active(ffn):
    """Which neurons the sparse layer's forward pass kept (its hybrid's entries), or None for the dense one."""
    import torch
    import unstructured_sparse_transformer_amd as tw
    if not hasattr(ffn, "hy"):
        return None
    h = torch.empty((ffn.hy.ell.T, ffn.hy.ell.F), dtype=torch.bfloat16, device="cuda")
    tw.twell_hybrid_to_dense(ffn.hy, h)
    return (h > 0).double().cpu()


def _reference(stack, x, dn):
    """Gradients in 64 bits by torch.autograd on the CPU, from the layers' 16-bit weights."""
    import torch
    wide = lambda t: t.detach().double().cpu().requires_grad_(True)  # noqa: E731
    x = wide(x)
    mats = [[wide(w) for w in c] for c in stack.copies]
    w_pre, w_post, gate = ([wide(w) for w in ws] for ws in (stack.w_pre, stack.w_post, stack.gate))

    def norm(v, w):
        return v / torch.sqrt(v.pow(2).mean(1, keepdim=True) + 1e-6) * w

    stream, n = x, norm(x, w_pre[0])
    for k, (wg, wu, wd) in enumerate(mats):
        g = n @ wg.T
        active = _active(stack.ffn[k])
        a = g / (1 + torch.exp(-g)) if active is None else g * active
        y = (a * (n @ wu.T)) @ wd
        stream = stream + stack.alpha * gate[k] * norm(y, w_post[k])
        n = norm(stream, w_pre[k + 1])
    n.backward(dn.double().cpu())
    return n, x.grad, [[w.grad for w in m] for m in mats], *([w.grad for w in ws] for ws in (w_pre, w_post, gate))


@pytest.mark.parametrize("ffn", ["Gated", "Sparse"])
def test_gradients(example, ffn):
    """Activations and gradients pass through bf16 (unit rounding 2^-8 at most) about six times a layer; errors of one
    tensor are independent, so two layers stay within 2^-8 sqrt(12) = 1.4% in the 2-norm; 4% are allowed.  ReLU's
    slope jumps at 0, where the rounded input may lie on the other side: the reference takes the neurons that the
    forward pass kept."""
    import torch
    say(f"case train layer {ffn}")
    T, d, F = 130, 128, 512
    stack = example.Stack(T, d, F, 2, getattr(example, ffn))
    gen = torch.Generator(device="cuda").manual_seed(3)
    x, dn = (torch.randn((T, d), generator=gen, device="cuda") for _ in range(2))
    n = stack.forward(x)
    dx = stack.backward(dn)
    want = _reference(stack, x, dn)

    def near(got, ref, label):
        got = got.double().cpu()
        rel = float((got - ref).norm() / ref.norm())
        assert rel < 0.04, f"{label}: {rel:.3g}"

    near(n, want[0].detach(), "n")
    near(dx, want[1], "dx")
    for k in range(2):
        for name, got, ref in zip(("dwg", "dwu", "dwd"), stack.ffn[k].grads, want[2][k]):
            near(got, ref, f"layer {k} {name}")
        near(stack.dw_post[k], want[4][k], f"dw_post {k}")
        near(stack.dgate[k], want[5][k], f"dgate {k}")
    for k in range(3):
        near(stack.dw_pre[k], want[3][k], f"dw_pre {k}")


@pytest.mark.parametrize("ffn", ["Gated", "Sparse"])
@pytest.mark.parametrize("bits", [32, 8])
def test_it_learns(example, ffn, bits):
    import torch
    say(f"case train layer learns {ffn} {bits}")
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((256, 128), generator=gen, device="cuda")
    target = torch.tanh(x.roll(1, 1)) + 0.5 * x
    stack = example.Stack(256, 128, 512, 2, getattr(example, ffn), bits)
    losses = []
    for _ in range(40):
        diff = stack.forward(x).float() - target
        losses.append(float(diff.square().mean()))
        stack.backward(diff * (2 / diff.numel()))
        stack.update(2e-3)
    assert losses[-1] < 0.5 * losses[0], losses[::10]
    for masters, copies in zip(stack.matrices, stack.copies):
        for p, c in zip(masters, copies):
            assert torch.equal(p.bfloat16(), c)


def test_step_in_a_graph(example):
    """Forward, backward and the optimizer in a captured graph: every replay changes the weights as the same eager
    steps do."""
    import torch
    say("case train layer in a graph")
    gen = torch.Generator(device="cuda").manual_seed(5)
    x, dn = (torch.randn((192, 128), generator=gen, device="cuda") for _ in range(2))
    stacks = [example.Stack(192, 128, 256, 2, example.Gated, 8) for _ in range(2)]

    def step(stack):
        stack.forward(x)
        stack.backward(dn)
        stack.step_count = 6  # the captured step's constants are the graph's
        stack.update(1e-3)

    step(stacks[1])  # torch's products set themselves up outside the capture
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(stacks[1])
    torch.cuda.current_stream().wait_stream(side)
    step(stacks[0])
    for k in range(4):
        graph.replay()
        step(stacks[0])
        torch.cuda.synchronize()
        for a, b in zip(stacks[0].optimizer.tensors, stacks[1].optimizer.tensors):
            for name in ("p", "m", "v", "grad"):
                assert torch.equal(a[name], b[name]), f"replay {k}: {name}"
