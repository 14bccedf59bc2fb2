"""A small language model trained with the library's operators alone around
torch's activation and loss: embedding lookup with learned positions and
dropout, 4-bit linear layers whose weight gradients are the bf16 matrices Muon
reads, residual dropout, and the embedding gradients that AdamW reads.

    python examples/train_step.py [--steps 60] [--format mx|nv]

The data is synthetic: each next token is a fixed function of the current one,
so the loss falls from log(vocab) towards 0.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import matrix_optimizers_zero_gb300 as mo  # noqa: E402


class Fp4Linear:
    """y = x w^T with 4-bit operands in all three products; the output
    gradient is rounded stochastically. `grad` is the bf16 gradient of w."""

    def __init__(self, tokens, rows, cols, fmt):
        self.w = torch.randn(rows, cols, device="cuda") / cols ** 0.5
        self.grad = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
        self.momentum = torch.zeros_like(self.w)
        self.y = torch.empty(tokens, rows, dtype=torch.bfloat16, device="cuda")
        self.dx = torch.empty(tokens, cols, dtype=torch.bfloat16, device="cuda")
        shapes = dict(x=(tokens, cols), xt=(cols, tokens), w=(rows, cols), wt=(cols, rows), dy=(tokens, rows), dyt=(rows, tokens))
        self.q = {name: mo.Fp4Tensor(r, k, fmt) for name, (r, k) in shapes.items()}

    def forward(self, x):
        mo.fp4_quantize(self.w, self.q["w"], self.q["wt"])   # both orientations from one pass
        mo.fp4_quantize(x, self.q["x"], self.q["xt"])
        mo.fp4_product(self.q["x"], self.q["w"], self.y)
        return self.y

    def backward(self, dy, random):
        mo.fp4_quantize(dy, self.q["dy"], self.q["dyt"], stochastic=random)
        mo.fp4_product(self.q["dy"], self.q["wt"], self.dx)
        mo.fp4_product(self.q["dyt"], self.q["xt"], self.grad)
        return self.dx


class Model:
    def __init__(self, vocab=512, dim=256, ff=1024, seq=64, batch=32, fmt="nv", p=0.05, seed=1):
        n = seq * batch
        self.vocab, self.seq, self.n, self.p, self.seed = vocab, seq, n, p, seed
        self.table = torch.randn(vocab, dim, device="cuda") * 0.5
        self.positions = torch.randn(seq, dim, device="cuda") * 0.1
        self.up, self.down, self.head = (Fp4Linear(n, *s, fmt) for s in ((ff, dim), (dim, ff), (vocab, dim)))
        self.x = torch.empty(n, dim, dtype=torch.bfloat16, device="cuda")
        self.z, self.dh = torch.empty_like(self.x), torch.empty_like(self.x)
        self.tail = [(t, torch.empty_like(t), torch.zeros_like(t), torch.zeros_like(t)) for t in (self.table, self.positions)]
        self.workspaces = [mo.embed_grad_workspace(n, *t.shape) for t in (self.table, self.positions)]
        self.position_ids = torch.arange(seq, device="cuda").repeat(batch)
        self.mats = [(l.w, l.grad, l.momentum) for l in (self.up, self.down, self.head)]
        self.muon = mo.MuonParams(lr=0.02, wd=0.0)
        self.muon_ws = mo.muon_workspace(self.mats, self.muon)

    def step(self, tokens, targets, t):
        """One training step (t from 1); the loss as a device tensor."""
        drop_x = mo.Dropout(self.p, self.seed, offset=8 * t)
        drop_y = mo.Dropout(self.p, self.seed, offset=8 * t + 1)
        random = [mo.Random(self.seed, 8 * t + 2 + 2 * i) for i in range(3)]
        # forward
        mo.embed_lookup(self.table, tokens, self.x, add=self.positions, dropout=drop_x)
        a = self.up.forward(self.x)
        h = torch.relu(a)
        mo.dropout_apply(self.down.forward(h), self.z, drop_y, residual=self.x)
        logits = self.head.forward(self.z).float().requires_grad_()
        loss = torch.nn.functional.cross_entropy(logits, targets)
        # backward
        loss.backward()
        dz = self.head.backward(logits.grad.bfloat16(), random[0])
        mo.dropout_apply(dz, self.dh, drop_y)
        da = self.down.backward(self.dh, random[1]) * (a > 0)
        dx = self.up.backward(da, random[2]) + dz
        for ids, (_, grad, _, _), ws in zip((tokens, self.position_ids), self.tail, self.workspaces):
            mo.embed_grad(dx, ids, grad, ws, dropout=drop_x)
        # update
        mo.muon_owner_step(self.mats, self.muon, self.muon_ws)
        mo.adamw_tail_step(self.tail, mo.AdamWParams(lr=3e-3, wd=0.0, step=t))
        return loss.detach()


def train(steps=60, fmt="nv", seed=1, log=None):
    torch.manual_seed(seed)
    model = Model(fmt=fmt, seed=seed)
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
    ap.add_argument("--format", choices=("mx", "nv"), default="nv")
    args = ap.parse_args()
    train(args.steps, args.format, log=print)
