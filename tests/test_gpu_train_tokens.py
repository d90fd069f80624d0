"""The training example on tokens: embedding, layers (with their activations in 8 bits
too), log probabilities and one optimizer step together, its gradients against torch's
derivatives in 64 bits."""

import importlib.util
import math
import os
import sys

import pytest

from helpers import say

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FFNS = ["Gated", "GatedKept8", "Sparse"]


@pytest.fixture(scope="module")
def example(gpu_lib):
    spec = importlib.util.spec_from_file_location("train_layer", os.path.join(ROOT, "examples", "train_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _batch(T, V, seed=0):
    """Tokens and the ones after them, padding among both."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ids, targets = (torch.randint(-1, V, (T,), generator=gen, device="cuda") for _ in range(2))
    ids[: T // 4] = 3  # one token has a quarter of the batch
    return ids, targets, torch.randn(T, generator=gen, device="cuda") / T


def _reference(model, ids, targets, dlogp):
    """Log probabilities and gradients in 64 bits by torch.autograd on the CPU, from the 16-bit weights."""
    import torch
    import unstructured_sparse_transformer_amd as tw
    stack = model.stack
    wide = lambda t: t.detach().double().cpu().requires_grad_(True)  # noqa: E731
    table, mats = wide(model.copy), [[wide(w) for w in c] for c in stack.copies]
    w_pre, w_post, gate = ([wide(w) for w in ws] for ws in (stack.w_pre, stack.w_post, stack.gate))
    ids, targets = ids.cpu(), targets.cpu()

    def norm(v, w):
        return v / torch.sqrt(v.pow(2).mean(1, keepdim=True) + 1e-6) * w

    stream = model.scale * table[ids.clamp_min(0)] * (ids >= 0)[:, None]
    n = norm(stream, w_pre[0])
    for k, (wg, wu, wd) in enumerate(mats):
        g = n @ wg.T
        if hasattr(stack.ffn[k], "hy"):  # ReLU, on the neurons that the forward pass kept
            h = torch.empty((model.T, wg.shape[0]), dtype=torch.bfloat16, device="cuda")
            tw.twell_hybrid_to_dense(stack.ffn[k].hy, h)
            a = g * (h > 0).double().cpu()
        else:
            a = g / (1 + torch.exp(-g))
        stream = stream + stack.alpha * gate[k] * norm((a * (n @ wu.T)) @ wd, w_post[k])
        n = norm(stream, w_pre[k + 1])
    logp = torch.log_softmax(n @ table.T, 1).gather(1, targets.clamp_min(0)[:, None])[:, 0] * (targets >= 0)
    logp.backward(dlogp.double().cpu())
    return logp.detach(), table.grad, [[w.grad for w in m] for m in mats], [w.grad for w in w_pre], [w.grad for w in w_post]


@pytest.mark.parametrize("ffn", FFNS)
def test_gradients(example, ffn):
    """Activations and gradients pass through bf16 (2^-8 at most) about six times a layer and four times at the ends, the
    kept g and u through 8 bits (half a step is 2^-8 of a block's largest, at most 2^-6 of its typical value): errors of
    one tensor are independent, so two layers stay within sqrt(16 + 4 * 16) 2^-8 = 3.5% in the 2-norm; 6% are allowed.
    A log probability has the logits' roundings, 2^-8 of at most 4, the layers' errors of the rows (1.4%) times the
    logits' size of about 1: 0.1 are allowed."""
    import torch
    say(f"case train tokens {ffn}")
    T, d, F, V = 130, 128, 512, 300
    model = example.Tokens(T, d, F, 2, V, ffn=getattr(example, ffn))
    ids, targets, dlogp = _batch(T, V)
    logp = model.forward(ids, targets).double().cpu()
    model.backward(dlogp)
    want = _reference(model, ids, targets, dlogp)
    assert (logp - want[0]).abs().max() < 0.1
    assert not logp[targets.cpu() < 0].any()

    def near(got, ref, label):
        rel = float((got.double().cpu() - ref).norm() / ref.norm())
        assert rel < 0.06, f"{label}: {rel:.3g}"

    near(model.grad, want[1], "table")
    for k in range(2):
        for name, got, ref in zip(("dwg", "dwu", "dwd"), model.stack.ffn[k].grads, want[2][k]):
            near(got, ref, f"layer {k} {name}")
        near(model.stack.dw_post[k], want[4][k], f"dw_post {k}")
    for k in range(3):
        near(model.stack.dw_pre[k], want[3][k], f"dw_pre {k}")


def test_likely_tokens(example):
    import torch
    say("case train tokens, likely")
    model = example.Tokens(70, 64, 128, 1, 1000)
    ids, targets, _ = _batch(70, 1000)
    model.forward(ids, targets)
    idx, top = model.likely(6)
    order = torch.sort(model.logits.float(), dim=1, descending=True, stable=True).indices[:, :6]
    assert torch.equal(idx.long(), order)
    want = torch.log_softmax(model.logits.double(), 1).gather(1, order)
    assert (top.double() - want).abs().max() < 1e-5  # 1000 terms of fp32: below 1000 * 2^-24


@pytest.mark.parametrize("ffn", FFNS[:2])
@pytest.mark.parametrize("bits", [8, 32])
def test_step_in_a_graph(example, ffn, bits):
    """The whole step captured: every replay, on other tokens each time, changes the weights as the same eager steps do."""
    import torch
    say(f"case train tokens in a graph {ffn} {bits}")
    T, V = 192, 500
    models = [example.Tokens(T, 128, 256, 2, V, ffn=getattr(example, ffn), bits=bits) for _ in range(2)]
    ids, targets, dlogp = _batch(T, V)

    def step(m):
        m.forward(ids, targets)
        m.backward(dlogp)
        m.stack.step_count = 6  # the captured step's constants are the graph's
        m.update(1e-3)

    step(models[1])  # torch's products set themselves up outside the capture
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(models[1])
    torch.cuda.current_stream().wait_stream(side)
    step(models[0])
    for k in range(4):
        for old, new in zip((ids, targets, dlogp), _batch(T, V, seed=k + 1)):
            old.copy_(new)
        graph.replay()
        step(models[0])
        torch.cuda.synchronize()
        assert torch.equal(models[0].logp, models[1].logp)
        for a, b in zip(models[0].stack.optimizer.tensors, models[1].stack.optimizer.tensors):
            for name in ("p", "m", "v", "grad"):
                assert torch.equal(a[name], b[name]), f"replay {k}: {name}"


@pytest.mark.parametrize("args", [["--keep", "8"], ["--vocab", "300"], ["--vocab", "300", "--keep", "8", "--bits", "8"],
                                  ["--vocab", "301", "--ffn", "sparse"]], ids=lambda a: "_".join(a).replace("--", ""))
def test_it_runs(example, args, monkeypatch, capsys):
    say(f"case train example {args}")
    monkeypatch.setattr(sys, "argv", ["train_layer.py", "--steps", "3", "--sizes", "100", "64", "256", "2", *args])
    example.main()
    lines = [x for x in capsys.readouterr().out.splitlines() if x.startswith("step")]
    assert len(lines) == 2 and all(math.isfinite(float(x.split()[3])) for x in lines)
