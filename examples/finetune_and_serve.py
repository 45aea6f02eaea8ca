"""Train a gated MLP block, fine-tune it for a few tasks, and serve all of them in
one batch: the variants' weights as low-rank adapters beside the packed base.

    python examples/finetune_and_serve.py [--steps 60] [--k 256] [--n 512] [--rank 8] [--tasks 3]

The block is Z = (SiLU(A W1) * (A W2)) W3 in bf16 with fp32 master weights.  Each
task moves the base by a fine-tuning run of its own; the truncated singular value
decomposition of what its weights moved by gives its adapters.  A batch whose rows
belong to different tasks then takes one packed call per product.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import swiglu_gated_mlp_amd as sw  # noqa: E402


def fit(masters, target, rows, steps, rate, seed, device):
    """Gradient steps of mean squared error towards target(A); returns (masters, losses)."""
    g = torch.Generator().manual_seed(seed)
    masters = [m.clone() for m in masters]
    losses = []
    for _ in range(steps):
        A = torch.randn(rows, masters[0].shape[0], generator=g).to(device).bfloat16()
        W = [m.bfloat16().requires_grad_() for m in masters]
        loss = (sw.swiglu_mlp(A, *W).float() - target(A)).square().mean()
        for m, grad in zip(masters, torch.autograd.grad(loss, W)):
            grad = grad.float()
            m -= rate * grad / (grad.square().mean().sqrt() + 1e-12)
        losses.append(loss.detach())
    return masters, [float(x) for x in losses]


def plain(A, W1, W2, W3):
    h = torch.nn.functional.silu(A.float() @ W1) * (A.float() @ W2)
    return h @ W3


def low_rank(change, rank):
    """(La, Lb) with La Lb near `change`, on the host."""
    u, s, v = torch.linalg.svd(change.float().cpu(), full_matrices=False)
    root = s[:rank].sqrt()
    return u[:, :rank] * root, root[:, None] * v[:rank]


def main(steps=60, K=256, N=512, rank=8, tasks=3, rows=512, device="cuda:0", out=print):
    g = torch.Generator().manual_seed(0)

    def weights(scale):
        return [scale * torch.randn(*s, generator=g).to(device) / s[0] ** 0.5 for s in ((K, N), (K, N), (N, K))]

    teacher = weights(1.0)
    base = [t + d for t, d in zip(teacher, weights(0.5))]
    base, losses = fit(base, lambda A: plain(A, *teacher), rows, steps, 2e-3, 1, device)
    out("base: loss %.4f -> %.4f" % (losses[0], losses[-1]))

    adapters = []
    for t in range(tasks):
        moved = [w + torch.randn(w.shape[0], 2, generator=g).to(device) @ torch.randn(2, w.shape[1], generator=g).to(
            device) * 0.5 / w.shape[0] ** 0.5 for w in teacher]
        tuned, task_losses = fit(base, lambda A: plain(A, *moved), rows, steps, 2e-3, 2 + t, device)
        adapters.append([low_rank(a - b, rank) for a, b in zip(tuned, base)])
        out("task %d: loss %.4f -> %.4f" % (t, task_losses[0], task_losses[-1]))

    # what a server holds: packed base weights, packed adapters, a scale per adapter
    W1, W2, W3 = (w.bfloat16() for w in base)
    Wp, W3g = sw.swiglu_pack_weights(W1, W2), sw.swiglu_gemm_pack_weight(W3)
    La, Lb = ([torch.stack([a[i][j] for a in adapters]).bfloat16().to(device) for i in range(3)] for j in range(2))
    Lp = sw.swiglu_lora_pack(La[0], Lb[0], La[1], Lb[1])
    Lp3 = sw.swiglu_gemm_lora_pack(La[2], Lb[2])
    scales = torch.ones(tasks, device=device)

    worst = 0.0
    for M in (1, 24, 200, 600):   # decode to prefill; task `tasks` stands for the base (no adapter)
        ids = torch.randint(0, tasks + 1, (M,), generator=g).to(device).int()
        ids[ids == tasks] = -1
        A = torch.randn(M, K, generator=g).to(device).bfloat16()
        Y = sw.swiglu_fused_packed_lora(A, Wp, Lp, ids, scales, N, rank)
        Z = sw.swiglu_gemm_packed_lora(Y, W3g, Lp3, ids, scales, K, rank)
        want = torch.empty_like(Z, dtype=torch.float32)
        for t in range(-1, tasks):
            merged = [w.float() if t < 0 else w.float() + La[i][t].float() @ Lb[i][t].float()
                      for i, w in enumerate((W1, W2, W3))]
            own = ids == t
            want[own] = plain(A[own], *merged)
        err = float((Z.float() - want).square().mean().sqrt() / want.square().mean().sqrt())
        out("served %4d rows of %d tasks: relative error against merged weights %.4f" % (M, tasks + 1, err))
        worst = max(worst, err)
    return losses, worst


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("steps", 60), ("k", 256), ("n", 512), ("rank", 8), ("tasks", 3)):
        p.add_argument("--" + name, type=int, default=default)
    a = p.parse_args()
    main(a.steps, a.k, a.n, a.rank, a.tasks)
