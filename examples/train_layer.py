"""Training steps of a small stack of feed-forward layers in the library's kernels.

    python examples/train_layer.py [--ffn gated|sparse] [--steps 50] [--bits 8|32] [--keep 8|16] [--vocab 4096]

A layer adds alpha * gate * norm(FFN(norm(stream))) to a 32-bit residual stream.  The norm after one FFN, the gate, the
sum and the norm before the next FFN are one call.  The FFN is the dense gated product followed by a plain matrix
product of torch's (``gated``; its backward pass takes two more), or the ReLU-sparse one on its hybrid activations
(``sparse``).  With ``--keep 8`` the gated FFN keeps its two products for the backward pass in 8 bits, and its hidden
activation not at all: all layers use one buffer for it.  The weights are 32-bit masters with 16-bit copies for the layers; one call updates all of them.

The layers learn a function of vectors, or with ``--vocab`` the token after each token: an embedding in front of them,
log probabilities behind them, and one table for both.
"""

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import unstructured_sparse_transformer_amd as tw  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


class Gated:
    """h = silu(n W_g) * (n W_u), y = h W_d.  first: the stack's first layer (None for that one itself)."""

    y_type = dx_type = BF16

    def __init__(self, T, d, F, weights, first=None):
        self.wg, self.wu, self.wd = weights
        new = lambda *s: torch.empty(s, dtype=BF16, device="cuda")  # noqa: E731
        self.h, self.g, self.u, self.y = new(T, F), new(T, F), new(T, F), new(T, d)
        self.dh, self.dx = new(T, F), new(T, d)
        self.grads = [new(F, d) for _ in range(3)]
        self.ws, self.ws_backward = tw.glu_workspace(T, d, F, BF16), tw.glu_backward_workspace(T, d, F, BF16)

    def forward(self, n):
        self.n = n
        tw.twell_glu_forward(n, self.wg, self.wu, "silu", self.h, self.ws, g=self.g, u=self.u)
        return torch.mm(self.h, self.wd, out=self.y)

    def backward(self, dy):
        torch.mm(dy, self.wd.t(), out=self.dh)
        torch.mm(self.h.t(), dy, out=self.grads[2])
        tw.twell_glu_backward(self.n, self.wg, self.wu, self.g, self.u, self.dh, "silu", self.dx, self.grads[0],
                              self.grads[1], self.ws_backward)
        return self.dx


class GatedKept8(Gated):
    """The same with g and u kept in 8 bits, and h taken from these again: what a layer keeps from its forward to its
    backward pass is these and y, and the layers of a stack share the buffers of h and dh and the workspaces."""

    def __init__(self, T, d, F, weights, first=None):
        self.wg, self.wu, self.wd = weights
        new = lambda *s: torch.empty(s, dtype=BF16, device="cuda")  # noqa: E731
        self.g, self.u = (tw.PackedAct.empty(T, F) for _ in range(2))
        self.y, self.dx, self.grads = new(T, d), new(T, d), [new(F, d) for _ in range(3)]
        if first is None:
            self.h, self.dh = new(T, F), new(T, F)
            self.ws, self.ws_backward = tw.glu_packed_workspace(T, d, F), tw.glu_backward_workspace(T, d, F, BF16)
        else:
            self.h, self.dh, self.ws, self.ws_backward = first.h, first.dh, first.ws, first.ws_backward

    def forward(self, n):
        self.n = n
        tw.twell_glu_forward_packed(n, self.wg, self.wu, "silu", self.h, self.g, self.u, self.ws)
        return torch.mm(self.h, self.wd, out=self.y)

    def backward(self, dy):
        torch.mm(dy, self.wd.t(), out=self.dh)
        tw.twell_glu_backward_packed(self.n, self.wg, self.wu, self.g, self.u, self.dh, "silu", self.dx, self.grads[0],
                                     self.grads[1], self.ws_backward, h=self.h)
        torch.mm(self.h.t(), dy, out=self.grads[2])
        return self.dx


class Sparse:
    """y = (ReLU(n W_g) * (n W_u)) W_d on the active neurons, forward and backward."""

    y_type = dx_type = F32

    def __init__(self, T, d, F, weights, first=None):
        self.wg, self.wu, self.wd = weights
        self.hy = tw.Hybrid.empty(T, F, 128, 32, BF16, T)
        self.y, self.dx = (torch.empty((T, d), dtype=F32, device="cuda") for _ in range(2))
        self.grads = [torch.empty((F, d), dtype=F32, device="cuda") for _ in range(3)]
        self.entries = T * F
        self.ws = tw.hybrid_workspace(self.hy, d)
        self.ws_backward = tw.backward_workspace(T, F, d, self.entries)

    def forward(self, n):
        self.n = n
        tw.twell_ffn_forward(n, self.wg, self.wu, self.wd, self.hy, self.y, self.ws)
        return self.y

    def backward(self, dy):
        tw.twell_ffn_backward(self.hy, self.n, self.wg, self.wu, self.wd, dy, self.dx, *self.grads, self.entries,
                              self.ws_backward)
        return self.dx


class Stack:
    """`layers` feed-forward layers between norms, their gradients and their optimizer."""

    def __init__(self, T, d, F, layers, ffn=Gated, bits=32, seed=0, alpha=0.5, others=()):
        """others: further tensors of the optimizer's step (p, copy, grad, weight_decay)."""
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
        self.T, self.alpha, self.step_count = T, alpha, 0
        self.matrices = [[rnd(F, d) * d ** -0.5, rnd(F, d) * d ** -0.5, rnd(F, d) * F ** -0.5] for _ in range(layers)]
        self.copies = [[w.to(BF16) for w in m] for m in self.matrices]
        ones = lambda: torch.ones(d, device="cuda")  # noqa: E731
        self.w_pre = [ones() for _ in range(layers + 1)]   # the norm before each FFN, and the last one
        self.w_post = [ones() for _ in range(layers)]      # the norm after each FFN
        self.gate = [ones().view(1, d) for _ in range(layers)]
        self.ffn = []
        for c in self.copies:
            self.ffn.append(ffn(T, d, F, c, *self.ffn[:1]))
        self.first = tw.BlockNorm(w_pre=self.w_pre[0])
        self.norms = [tw.BlockNorm(alpha=alpha, post=True, w_post=self.w_post[k], w_pre=self.w_pre[k + 1])
                      for k in range(layers)]
        row = lambda dt: torch.empty((T, d), dtype=dt, device="cuda")  # noqa: E731
        self.stream = [None] + [row(F32) for _ in range(layers)]
        self.n = [row(BF16) for _ in range(layers + 1)]
        self.dstream, self.dy, self.ws = row(F32), row(ffn.y_type), tw.block_norm_workspace(T, d)
        zeros = lambda t: torch.zeros_like(t)  # noqa: E731
        self.dw_pre, self.dw_post = [zeros(w) for w in self.w_pre], [zeros(w) for w in self.w_post]
        self.dgate = [zeros(g) for g in self.gate]
        sets = [dict(p=p, copy=c, grad=g, weight_decay=0.01)
                for m, cs, f in zip(self.matrices, self.copies, self.ffn) for p, c, g in zip(m, cs, f.grads)]
        sets += [dict(p=p, grad=g) for p, g in zip(self.w_pre + self.w_post + self.gate,
                                                   self.dw_pre + self.dw_post + self.dgate)]
        sets += [dict(t) for t in others]
        for t in sets:
            if bits == 8:
                blocks = -(-t["p"].numel() // tw.ADAMW_BLOCK)
                t.update(m=torch.zeros(t["p"].shape, dtype=torch.uint8, device="cuda"),
                         v=torch.zeros(t["p"].shape, dtype=torch.uint8, device="cuda"),
                         m_scale=torch.zeros(blocks, device="cuda"), v_scale=torch.zeros(blocks, device="cuda"))
            else:
                t.update(m=zeros(t["p"]), v=zeros(t["p"]))
        self.optimizer = tw.AdamWTensors(sets)

    def forward(self, x):
        """The normed output [T][d] bf16 of the stack for x [T][d] float."""
        self.stream[0] = x
        tw.twell_block_norm_forward(self.first, x, None, None, self.n[0])
        for k, (ffn, bn) in enumerate(zip(self.ffn, self.norms)):
            y = ffn.forward(self.n[k])
            tw.twell_block_norm_forward(bn, self.stream[k], y, self.stream[k + 1], self.n[k + 1], gate=self.gate[k],
                                        gate_span=self.T)
        return self.n[-1]

    def backward(self, dn):
        """Gradients of all weights, and of x (returned), from that of the output (float)."""
        dout = None
        for k in reversed(range(len(self.ffn))):
            ffn, bn = self.ffn[k], self.norms[k]
            tw.twell_block_norm_backward(bn, self.stream[k + 1], ffn.y, dout, dn, self.dstream, self.dy, self.ws,
                                         gate=self.gate[k], gate_span=self.T, dgate=self.dgate[k],
                                         dw_post=self.dw_post[k], dw_pre=self.dw_pre[k + 1])
            dout, dn = self.dstream, ffn.backward(self.dy)
        tw.twell_block_norm_backward(self.first, self.stream[0], None, dout, dn, self.dstream, None, self.ws,
                                     dw_pre=self.dw_pre[0])
        return self.dstream

    def update(self, lr):
        self.step_count += 1
        tw.twell_adamw_step(self.optimizer, lr, 0.9, 0.95, 1e-8, self.step_count, seed=self.step_count)


class Tokens:
    """The stack between a table's rows for tokens (ids [T], int64; -1: padding) and log probabilities of the tokens after
    them, from products with the same rows."""

    def __init__(self, T, d, F, layers, V, seed=0, **stack):
        gen = torch.Generator(device="cuda").manual_seed(seed + 100)
        self.table = torch.randn((V, d), generator=gen, device="cuda") * d ** -0.5
        self.copy, self.grad = self.table.to(BF16), torch.empty((V, d), dtype=BF16, device="cuda")
        self.stack = Stack(T, d, F, layers, seed=seed, others=[dict(p=self.table, copy=self.copy, grad=self.grad)], **stack)
        new = lambda *s, dt=F32: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
        self.T, self.scale = T, math.sqrt(d)
        self.x, self.logits, self.dn = new(T, d), new(T, V, dt=BF16), new(T, d, dt=BF16)
        self.logp, self.norm = new(T), new(T, 2)
        self.ws, self.ws_backward = tw.logprob_workspace(T, V), tw.embed_workspace(T, V, d)

    def forward(self, ids, targets):
        """The log probabilities [T] of the targets (0 where one is -1)."""
        self.ids, self.targets = ids, targets
        tw.twell_embed_forward(ids, self.copy, self.x, scale=self.scale)
        self.n = self.stack.forward(self.x)
        torch.mm(self.n, self.copy.t(), out=self.logits)
        tw.twell_logprob_forward(self.logits, targets, self.logp, self.norm, self.ws)
        return self.logp

    def backward(self, dlogp):
        """Gradients of all weights from that of the log probabilities; the logits make place for theirs."""
        tw.twell_logprob_backward(self.logits, self.targets, self.norm, dlogp, self.logits)
        torch.mm(self.logits, self.copy, out=self.dn)
        torch.mm(self.logits.t(), self.n, out=self.grad)
        dx = self.stack.backward(self.dn)
        tw.twell_embed_backward(self.ids, dx, self.grad, self.ws_backward, scale=self.scale, accumulate=True)

    def update(self, lr):
        self.stack.update(lr)

    def likely(self, k):
        """The k most likely tokens after each, after forward and before backward."""
        idx = torch.empty((self.T, k), dtype=torch.int32, device="cuda")
        top = torch.empty((self.T, k), device="cuda")
        tw.twell_logprob_forward(self.logits, None, None, None, tw.logprob_workspace(*self.logits.shape, k), top_logp=top,
                                 top_idx=idx)
        return idx, top


def train_tokens(a, ffn):
    T, d, F, layers = a.sizes
    gen = torch.Generator(device="cuda").manual_seed(1)
    after = torch.randperm(a.vocab, generator=gen, device="cuda")  # the token after each token, to be learned
    model = Tokens(T, d, F, layers, a.vocab, ffn=ffn, bits=a.bits)
    dlogp = torch.full((T,), -1 / T, device="cuda")
    for step in range(a.steps):
        u = torch.rand(T, generator=gen, device="cuda", dtype=torch.float64)
        ids = (torch.exp(u * math.log(a.vocab + 1)).long() - 1).clamp(0, a.vocab - 1)  # few tokens are most of a text
        loss = -model.forward(ids, after[ids]).mean()
        hits = None
        if step % 10 == 0 or step + 1 == a.steps:
            hits = (model.likely(1)[0][:, 0] == after[ids]).float().mean()
        model.backward(dlogp)
        model.update(2e-3)
        if hits is not None:
            print(f"step {step:4d}  loss {loss.item():.5f}  most likely token right {hits.item():.3f}", flush=True)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--ffn", choices=("gated", "sparse"), default="gated")
    ap.add_argument("--bits", type=int, choices=(8, 32), default=32)
    ap.add_argument("--keep", type=int, choices=(8, 16), default=16)
    ap.add_argument("--vocab", type=int, default=0)
    ap.add_argument("--steps", type=int, default=50)
    ap.add_argument("--sizes", type=int, nargs=4, default=(512, 256, 1024, 2), metavar=("T", "d", "F", "layers"))
    a = ap.parse_args()
    if a.keep == 8 and a.ffn != "gated":
        ap.error("--keep 8 is the gated FFN's")
    ffn = GatedKept8 if a.keep == 8 else {"gated": Gated, "sparse": Sparse}[a.ffn]
    if a.vocab:
        train_tokens(a, ffn)
        return
    T, d, F, layers = a.sizes
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((T, d), generator=gen, device="cuda")
    target = torch.tanh(x.roll(1, 1)) + 0.5 * x  # a mixing of neighbouring channels, to be learned
    stack = Stack(T, d, F, layers, ffn, a.bits)
    for step in range(a.steps):
        diff = stack.forward(x).float() - target
        stack.backward(diff * (2 / diff.numel()))
        stack.update(2e-3)
        if step % 10 == 0 or step + 1 == a.steps:
            print(f"step {step:4d}  loss {diff.square().mean().item():.5f}", flush=True)


if __name__ == "__main__":
    main()
