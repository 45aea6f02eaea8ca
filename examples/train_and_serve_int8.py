"""Train a gated MLP block with its checkpoints in 8 bits, then serve it in 8 bits.

    python examples/train_and_serve_int8.py [--steps 60] [--k 256] [--n 512] [--rows 512]

The block is Z = (SiLU(A W1) * (A W2)) W3 in bf16 with fp32 master weights.  Between
its forward and backward pass Gate and Up are kept as int8 with a scale for each 32
columns of a row; the trained weights then get a scale for each column and are packed
once, and the rows of a batch are quantized as they come.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import swiglu_gated_mlp_amd as sw  # noqa: E402


def gradients(A, target, W):
    """Mean squared error of the block on A against target, and its gradients by W."""
    W = [w.detach().requires_grad_() for w in W]
    loss = (sw.swiglu_mlp(A, *W, keep="int8").float() - target).square().mean()
    return loss.detach(), torch.autograd.grad(loss, W)


def plain(A, W1, W2, W3):
    h = torch.nn.functional.silu(A.float() @ W1.float()) * (A.float() @ W2.float())
    return h @ W3.float()


class Served:
    """What a server holds of a block: packed codes, their columns' scales, a workspace."""

    def __init__(self, W1, W2, W3):
        (q1, self.s1), (q2, self.s2), (q3, self.s3) = (sw.swiglu_quantize_columns_int8(w) for w in (W1, W2, W3))
        self.Wp, self.W3g = sw.swiglu_pack_weights_int8(q1, q2), sw.swiglu_gemm_pack_weight_int8(q3)
        self.workspace = sw.Workspace(W1.device)

    def __call__(self, A):
        return sw.swiglu_mlp_packed_int8(A, self.Wp, self.s1, self.s2, self.W3g, self.s3, workspace=self.workspace)[1]


def main(steps=60, K=256, N=512, rows=512, device="cuda:0", out=print):
    g = torch.Generator().manual_seed(0)

    def weights(scale):
        return [scale * torch.randn(*s, generator=g).to(device) / s[0] ** 0.5 for s in ((K, N), (K, N), (N, K))]

    teacher = weights(1.0)
    masters = [t + d for t, d in zip(teacher, weights(0.5))]
    losses = []
    for _ in range(steps):
        A = torch.randn(rows, K, generator=g).to(device).bfloat16()
        loss, grads = gradients(A, plain(A, *teacher), [m.bfloat16() for m in masters])
        for m, grad in zip(masters, grads):
            grad = grad.float()
            m -= 2e-3 * grad / (grad.square().mean().sqrt() + 1e-12)
        losses.append(loss)
    out("loss %.4f -> %.4f" % (float(losses[0]), float(losses[-1])))

    W = [m.bfloat16() for m in masters]
    served, worst = Served(*W), 0.0
    for M in (1, 24, 200, 600):   # decode to prefill
        A = torch.randn(M, K, generator=g).to(device).bfloat16()
        Z, want = served(A).float(), plain(A, *W)
        err = float((Z - want).square().mean().sqrt() / want.square().mean().sqrt())
        out("served %4d rows: relative error against the block in bf16 %.4f" % (M, err))
        worst = max(worst, err)
    return W, worst


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("steps", 60), ("k", 256), ("n", 512), ("rows", 512)):
        p.add_argument("--" + name, type=int, default=default)
    a = p.parse_args()
    main(a.steps, a.k, a.n, a.rows)
