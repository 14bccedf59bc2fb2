"""A small language model whose layers are the library's feed-forward operators,
with activation checkpoints in 8 bits: a Llama-style gated block, a GPT-2 style
block of two products, and a head, trained with Muon and AdamW. Embeddings are
the library's too; torch computes the loss.

    python examples/feed_forward_step.py [--steps 60]

The data is synthetic: each next token is a fixed function of the current one.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import matrix_optimizers_zero_gb300 as mo  # noqa: E402

BF16 = torch.bfloat16


def empty(*shape, dtype=BF16):
    return torch.empty(shape, dtype=dtype, device="cuda")


class Matrix:
    """An fp32 weight, the bf16 copy that products read, and what Muon reads and keeps."""

    def __init__(self, rows, cols):
        self.w = torch.randn(rows, cols, device="cuda") / cols ** 0.5
        self.b = self.w.to(BF16)
        self.grad, self.momentum = empty(rows, cols), torch.zeros_like(self.w)

    def refresh(self):
        self.b.copy_(self.w)


class Vector:
    """An fp32 weight or bias and what AdamW reads and keeps."""

    def __init__(self, value):
        self.w = value
        self.grad, self.m, self.v = torch.empty_like(value), torch.zeros_like(value), torch.zeros_like(value)

    def tail(self):
        return self.w, self.grad, self.m, self.v


class GatedBlock:
    """s += gated_ffn(norm(s)); all that its backward pass keeps is in 8 bits."""

    def __init__(self, n, dim, inner):
        self.norm = Vector(torch.ones(dim, device="cuda"))
        self.gate, self.up, self.down = Matrix(inner, dim), Matrix(inner, dim), Matrix(dim, inner)
        self.s8, self.n8 = mo.Mx8Tensor(n, dim), mo.Mx8Tensor(n, dim)
        self.g8, self.u8 = mo.Mx8Tensor(n, inner), mo.Mx8Tensor(n, inner)
        self.dn = empty(n, dim)
        self.matrices, self.vectors = [self.gate, self.up, self.down], [self.norm]

    def forward(self, s, ws):
        mo.mx8_quantize(s, self.s8)
        mo.rms_norm(s, weight=self.norm.w, out8=self.n8)
        mo.gated_ffn(self.n8, self.gate.b, self.up.b, self.down.b, s, residual=s, gate=self.g8, up=self.u8, workspace=ws)

    def backward(self, ds, ws, norm_ws):
        mo.gated_ffn_grad(ds, self.n8, self.g8, self.u8, self.gate.b, self.up.b, self.down.b, dx=self.dn, dw_gate=self.gate.grad,
                          dw_up=self.up.grad, dw_down=self.down.grad, workspace=ws)
        mo.rms_norm_grad(self.dn, self.s8, ds, weight=self.norm.w, dresidual=ds, dweight=self.norm.grad, workspace=norm_ws)


class PlainBlock:
    """s += w2 gelu(w1 norm(s) + b1) + b2; the stream and the activation's argument are kept in 8 bits."""

    def __init__(self, n, dim, inner):
        self.norm, self.b1, self.b2 = (Vector(v) for v in (torch.ones(dim, device="cuda"), torch.zeros(inner, device="cuda"),
                                                           torch.zeros(dim, device="cuda")))
        self.w1, self.w2 = Matrix(inner, dim), Matrix(dim, inner)
        self.s8, self.z8 = mo.Mx8Tensor(n, dim), mo.Mx8Tensor(n, inner)
        self.n, self.h, self.dn, self.dh = empty(n, dim), empty(n, inner), empty(n, dim), empty(n, inner)
        self.matrices, self.vectors = [self.w1, self.w2], [self.norm, self.b1, self.b2]

    def forward(self, s, ws):
        mo.mx8_quantize(s, self.s8)
        mo.rms_norm(s, self.n, weight=self.norm.w)
        mo.linear(self.n, self.w1.b, self.h, bias=self.b1.w, activation="gelu_tanh", pre=self.z8, workspace=ws)
        mo.linear(self.h, self.w2.b, s, bias=self.b2.w, residual=s, workspace=ws)

    def backward(self, ds, ws, norm_ws):
        mo.linear_grad(ds, self.h, self.w2.b, dx=self.dh, dw=self.w2.grad, dbias=self.b2.grad, workspace=ws)
        mo.linear_grad(self.dh, self.n, self.w1.b, dx=self.dn, dw=self.w1.grad, dbias=self.b1.grad, activation="gelu_tanh", pre=self.z8,
                       workspace=ws)
        mo.rms_norm_grad(self.dn, self.s8, ds, weight=self.norm.w, dresidual=ds, dweight=self.norm.grad, workspace=norm_ws)


class Model:
    def __init__(self, vocab=512, dim=256, inner=704, seq=64, batch=32, seed=1):
        torch.manual_seed(seed)
        n = seq * batch
        self.vocab, self.n = vocab, n
        self.table = Vector(torch.randn(vocab, dim, device="cuda") * 0.5)
        self.blocks = [GatedBlock(n, dim, inner), PlainBlock(n, dim, inner)]
        self.norm, self.head = Vector(torch.ones(dim, device="cuda")), Matrix(vocab, dim)
        self.s, self.z, self.ds, self.dz = (empty(n, dim) for _ in range(4))
        self.logits = empty(n, vocab, dtype=torch.float32)
        # one workspace for all of them: the calls of a step run one after the other
        sizes = [mo.mo_gated_ffn_workspace_bytes(n, dim, inner, grad=True)]
        sizes += [mo.mo_linear_workspace_bytes(n, cols, rows, grad=True) for cols, rows in ((dim, inner), (inner, dim), (dim, vocab))]
        self.ws = empty(max(sizes), dtype=torch.uint8)
        self.norm_ws = mo.rms_norm_grad_workspace(n, dim)
        self.embed_ws = mo.embed_grad_workspace(n, vocab, dim)
        self.matrices = [m for b in self.blocks for m in b.matrices] + [self.head]
        self.tail = [v.tail() for v in [self.table, self.norm] + [v for b in self.blocks for v in b.vectors]]
        self.muon = mo.MuonParams(lr=0.02, wd=0.0)
        self.mats = [(m.w, m.grad, m.momentum) for m in self.matrices]
        self.muon_ws = mo.muon_workspace(self.mats, self.muon)

    def forward(self, tokens):
        mo.embed_lookup(self.table.w, tokens, self.s)
        for b in self.blocks:
            b.forward(self.s, self.ws)
        mo.rms_norm(self.s, self.z, weight=self.norm.w)
        mo.linear(self.z, self.head.b, self.logits, workspace=self.ws)

    def backward(self, tokens, dlogits):
        mo.linear_grad(dlogits, self.z, self.head.b, dx=self.dz, dw=self.head.grad, workspace=self.ws)
        mo.rms_norm_grad(self.dz, self.s, self.ds, weight=self.norm.w, dweight=self.norm.grad, workspace=self.norm_ws)
        for b in reversed(self.blocks):
            b.backward(self.ds, self.ws, self.norm_ws)
        mo.embed_grad(self.ds, tokens, self.table.grad, self.embed_ws)

    def step(self, tokens, targets, t):
        """One training step (t from 1); the loss as a device tensor."""
        self.forward(tokens)
        logits = self.logits.detach().requires_grad_()
        loss = torch.nn.functional.cross_entropy(logits, targets)
        loss.backward()
        self.backward(tokens, logits.grad.to(BF16))
        mo.muon_owner_step(self.mats, self.muon, self.muon_ws)
        mo.adamw_tail_step(self.tail, mo.AdamWParams(lr=3e-3, wd=0.0, step=t))
        for m in self.matrices:
            m.refresh()
        return loss.detach()


def train(steps=60, seed=1, log=None):
    model = Model(seed=seed)
    follow = torch.randperm(model.vocab, device="cuda")   # each token's successor
    losses = []
    for t in range(1, steps + 1):
        tokens = torch.randint(0, model.vocab, (model.n,), device="cuda")
        losses.append(model.step(tokens, follow[tokens], t))
        if log and (t == 1 or t % 10 == 0):
            log(f"step {t:4d}  loss {losses[-1].item():.4f}")
    status = mo.mo_last_device_error()
    if status != 0:
        raise RuntimeError(mo.mo_status_string(status))
    return [float(x) for x in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    train(ap.parse_args().steps, log=print)
