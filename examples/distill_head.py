#!/usr/bin/env python3
"""A head on looked-up rows, distilled from a teacher's top logits.

    bags -> pooled rows (TT table) -> layer norm -> gated block -> class logits

Trains the table's cores and the head together, one training step a batch:
forward and backward of every operator by the library, the plain product with
the classes' matrix and its gradients by torch. Then answers a single bag the
way a server would. Every buffer is allocated once, before the loop.

    python3 examples/distill_head.py [--batch 256] [--steps 100] [--dtype bf16]
"""
import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import torch  # noqa: E402

import tensor_train_compressed_amd as tte  # noqa: E402
import workloads as wl  # noqa: E402

DEV = "cuda:0"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


class Table:
    """The TT table's cores on the device, and the plan of one batch of bags."""

    def __init__(self, problem):
        self.shapes = tte.make_tables(problem.tables, problem.goff)
        self.cores = [torch.from_numpy(c).to(DEV) for c in (problem.g1, problem.g2, problem.g3)]
        self.dim = problem.dim

    def plan(self, indices, offsets):
        return tte.tt_emb_plan(self.shapes, indices, offsets, offsets.numel() - 1, 256)


class Head:
    """Layer norm, gated block and classes' matrix, with their gradients'
    buffers and the workspaces for batches of up to `rows` bags."""

    def __init__(self, rows, dim, hidden, classes, dtype, act="silu", seed=0):
        g = torch.Generator(device=DEV).manual_seed(seed)

        def weight(n, k):
            return (torch.randn(n, k, generator=g, device=DEV) / k ** 0.5).to(dtype)

        self.dtype, self.act = dtype, act
        self.params = {"norm_weight": torch.ones(dim, device=DEV), "norm_bias": torch.zeros(dim, device=DEV),
                       "w_gate": weight(hidden, dim), "w_up": weight(hidden, dim), "classes": weight(classes, hidden)}
        self.grads = {k: torch.empty_like(v) for k, v in self.params.items()}
        f32 = dict(dtype=torch.float32, device=DEV)
        t = dict(dtype=dtype, device=DEV)
        self.x, self.y, self.dy, self.dx = (torch.empty(rows, dim, **t) for _ in range(4))
        self.mean, self.rstd = torch.empty(rows, **f32), torch.empty(rows, **f32)
        self.gate, self.up = torch.empty(rows, hidden, **f32), torch.empty(rows, hidden, **f32)
        self.out, self.dout = torch.empty(rows, hidden, **t), torch.empty(rows, hidden, **t)
        self.logits, self.dlogits = torch.empty(rows, classes, **t), torch.empty(rows, classes, **t)
        self.loss = torch.empty(rows, **f32)
        need = max(tte.tt_emb_norm_workspace_bytes(dtype, rows, dim),
                   tte.tt_emb_gate_workspace_bytes(dtype, rows, dim, hidden),
                   tte.tt_emb_distill_workspace_bytes(dtype, rows, classes))
        self.workspace = torch.empty(need, dtype=torch.uint8, device=DEV)   # one: the calls follow each other

    def forward(self, pooled, keep):
        """Logits of pooled rows [n, dim] (n up to the buffers' rows); `keep`: what the backward needs is kept."""
        n, p = pooled.shape[0], self.params
        x, y, out, logits = self.x[:n], self.y[:n], self.out[:n], self.logits[:n]
        x.copy_(pooled)
        kept = (self.mean[:n], self.rstd[:n]) if keep else (None, None)
        tte.tt_emb_norm_forward(x, p["norm_weight"], p["norm_bias"], y, *kept)
        kept = (self.gate[:n], self.up[:n]) if keep else (None, None)
        tte.tt_emb_gate_forward(y, p["w_gate"], p["w_up"], out, *kept, act=self.act, workspace=self.workspace)
        return torch.mm(out, p["classes"].t(), out=logits)

    def backward(self, n):
        """Every parameter's gradient, and the pooled rows' (returned), from self.dlogits."""
        p, g = self.params, self.grads
        dlogits, dout, dy, dx = self.dlogits[:n], self.dout[:n], self.dy[:n], self.dx[:n]
        torch.mm(dlogits.t(), self.out[:n], out=g["classes"])
        torch.mm(dlogits, p["classes"], out=dout)
        tte.tt_emb_gate_backward(self.y[:n], p["w_gate"], p["w_up"], self.gate[:n], self.up[:n], dout, dy, g["w_gate"],
                                 g["w_up"], act=self.act, workspace=self.workspace)
        tte.tt_emb_norm_backward(self.x[:n], p["norm_weight"], self.mean[:n], self.rstd[:n], dy, dx, g["norm_weight"],
                                 g["norm_bias"], workspace=self.workspace)
        return dx

    def sgd(self, lr):
        for k, v in self.params.items():
            v.add_(self.grads[k], alpha=-lr)


def train_step(table, head, plan, pooled, ids, top_logits, row_weight, temperature, lr, table_lr):
    """One step on the plan's batch; returns the rows' losses (before the step)."""
    kept = tte.tt_emb_forward_train(plan, *table.cores, pooled)
    logits = head.forward(pooled, keep=True)
    n = pooled.shape[0]
    tte.tt_emb_distill_train(logits, ids, top_logits, row_weight, head.loss[:n], head.dlogits[:n],
                             temperature=temperature, workspace=head.workspace)
    dpooled = head.backward(n).float()
    tte.tt_emb_backward_sgd(plan, kept, *table.cores, dpooled, table_lr)
    head.sgd(lr)
    return head.loss[:n]


def answer(table, head, indices, offsets, pooled, top):
    """The top classes of each bag and their logits."""
    plan = table.plan(indices, offsets)
    tte.tt_emb_forward(plan, *table.cores, pooled)
    return torch.topk(head.forward(pooled, keep=False), top, dim=1)


def teacher_lists(bags, classes, top, seed):
    """A stand-in teacher: each bag's classes follow from its number, a few lists are cut short."""
    g = torch.Generator().manual_seed(seed)
    start = (torch.arange(bags) * 7919) % classes
    ids = (start[:, None] + 13 * torch.arange(top)) % classes
    top_logits = 6.0 - 0.3 * torch.rand(bags, top, generator=g).cumsum(1)
    ids[torch.rand(bags, 1, generator=g).expand(-1, top) < 0.05] = -1    # no list: no loss, no gradient
    return ids.to(DEV), top_logits.to(DEV)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--batch", type=int, default=256)
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--classes", type=int, default=1000)
    ap.add_argument("--steps", type=int, default=100)
    ap.add_argument("--dtype", choices=list(DTYPES), default="bf16")
    a = ap.parse_args()
    p = wl.make("train11m", batch=a.batch)
    table = Table(p)
    indices, offsets = torch.from_numpy(p.indices).to(DEV), torch.from_numpy(p.offsets).to(DEV)
    head = Head(a.batch, p.dim, a.hidden, a.classes, DTYPES[a.dtype])
    ids, top_logits = teacher_lists(a.batch, a.classes, 16, seed=1)
    row_weight = torch.full((a.batch,), 1.0 / a.batch, device=DEV)   # the mean loss
    pooled = torch.empty(a.batch, p.dim, device=DEV)
    plan = table.plan(indices, offsets)
    for step in range(a.steps):
        loss = train_step(table, head, plan, pooled, ids, top_logits, row_weight, 2.0, lr=0.5, table_lr=0.05)
        if step % 10 == 0 or step == a.steps - 1:
            print(f"step {step}: mean loss {float(loss.mean()):.4f}", flush=True)
    one = offsets[:2]
    top = answer(table, head, indices[:int(one[1])].contiguous(), one.contiguous(), pooled[:1], 5)
    print("bag 0 answers", top.indices[0].tolist(), "of the teacher's", ids[0, :5].tolist())


if __name__ == "__main__":
    main()
