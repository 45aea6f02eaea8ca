"""The gated MLP in 8-bit integers, as it is measured: products of int8 operands
for serving, and int8 checkpoints of Gate and Up for training.

Every case is one pass on bf16 activations on the GPU:

  product   A's rows quantized to int8, then Y = SiLU(G) * U with G = A W1, U = A W2
            of int8 weights with a scale for each column
  down      the same with one weight: C = A W
  mlp       the whole block: Y as in product, then Z = Y W3 with Y's rows quantized
  step      one training step's forward and backward pass of Y = SiLU(G) * U: G and
            U are kept between the two as int8 with a scale for 32 columns of a row
  block     the backward pass of Z = Y W3 from dZ with G and U kept that way and Y
            computed from them: dA, dW1, dW2, dW3

Quantized rows (columns, groups of 32) x have the scale s = max |x| / 127 and hold
round(x / s); the scales of kept G and U are bf16, rounded up.

``own`` False computes them in fp32 with elementary torch operations, ``own`` True
through swiglu_gated_mlp_amd.  The widths are the repository's workloads (K x N of
the gate/up projections 896 x 4864, 3584 x 18944 and 8192 x 29568) and odd ones
between them.
"""
from __future__ import annotations

import math

import torch

own = False

_BF16 = torch.bfloat16
_TINY = 2.0 ** -96      # the least maximum a row's scale is made from


def listed():
    return [
        # one request's next token; a decode batch at the largest width; a prompt
        # batch, bound by the matrix cores
        dict(name="product-7b-m1", op="product", M=1, K=3584, N=18944),
        dict(name="product-72b-m32", op="product", M=32, K=8192, N=29568),
        dict(name="product-7b-m8192", op="product", M=8192, K=3584, N=18944),
        # the down projection alone: a decode batch (a long contraction to few
        # columns), and a ragged batch at a width that no tile divides
        dict(name="down-7b-m16", op="down", M=16, K=18944, N=3584),
        dict(name="down-odd-m777", op="down", M=777, K=5904, N=1416),
        # the whole block: a decode batch at the smallest width (latency), one that
        # is too large for the decode schedule, a prompt batch
        dict(name="mlp-0.5b-m64", op="mlp", M=64, K=896, N=4864),
        dict(name="mlp-7b-m128", op="mlp", M=128, K=3584, N=18944),
        dict(name="mlp-7b-m4096", op="mlp", M=4096, K=3584, N=18944),
        # training with int8 checkpoints: a last, short micro-batch at the smallest
        # width, and a training batch at the 7B width
        dict(name="step-0.5b-m333", op="step", M=333, K=896, N=4864),
        dict(name="step-7b-m4096", op="step", M=4096, K=3584, N=18944),
        # the block's backward pass: a ragged batch at an odd width, and 2048 tokens
        dict(name="block-odd-m1003", op="block", M=1003, K=1416, N=5896),
        dict(name="block-7b-m2048", op="block", M=2048, K=3584, N=18944),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the listed ones' ranges: widths from 128 x 256 to the 72B one, 1 to
    8192 rows, no dearer than the 4096-row training step."""
    op = rng.choice(["product", "product", "down", "down", "mlp", "mlp", "step", "block"])
    limit = 12 * 4096 * 3584 * 18944
    while True:
        M = _log_int(rng, 1, 8192)
        if op in ("step", "block"):
            K, N = 8 * _log_int(rng, 16, 1024), 8 * _log_int(rng, 32, 3696)
        else:
            K, N = 16 * _log_int(rng, 8, 512), 16 * _log_int(rng, 16, 1848)
        if op == "down":
            K, N = N, K
        case = dict(op=op, M=M, K=K, N=N)
        # tiny widths with a handful of rows would only time the launch
        if work(case)["flops"] <= limit and K * N >= 1 << 18:
            return case


def _normal(gen, *shape, std=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(_BF16)


def _activations(gen, M, K):
    """Normalised activations: rows of differing size, a few large channels."""
    a = torch.randn(M, K, generator=gen, device="cuda")
    a *= torch.exp(0.3 * torch.randn(M, 1, generator=gen, device="cuda"))
    big = torch.randint(0, K, (max(1, K // 256),), generator=gen, device="cuda")
    a[:, big] *= 6.0
    return a.to(_BF16)


def _weight8(gen, K, N):
    """An int8 weight and its columns' scales, as a quantized checkpoint holds them."""
    w = torch.randn(K, N, generator=gen, device="cuda") * K ** -0.5
    top = w.abs().amax(0)
    return torch.round(w * (127.0 / top)).to(torch.int8), top / 127.0


def _checkpoint(g, u):
    """Codes [M, groups, 2, 32] int8 and scales [groups, M, 2] bf16 of Gate and Up."""
    M, N = g.shape
    groups = (N + 31) // 32
    x = torch.zeros(2, M, groups * 32, device=g.device)
    x[0, :, :N], x[1, :, :N] = g, u
    x = x.view(2, M, groups, 32)
    # bf16 rounded up: the low half of the bits carried into the upper one
    s = ((x.abs().amax(3) / 127.0).view(torch.int32) + 0xFFFF) >> 16 << 16
    s = s.view(torch.float32).clamp_min(2.0 ** -126)
    codes = torch.round(x / s[..., None]).to(torch.int8)
    return codes.permute(1, 2, 0, 3).contiguous(), s.to(_BF16).permute(2, 1, 0).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op, M, K, N = case["op"], case["M"], case["K"], case["N"]
    st = {"case": dict(case)}
    if op in ("step", "block"):
        st["A"] = _normal(gen, M, K)
        st["W1"] = _normal(gen, K, N, std=K ** -0.5)
        st["W2"] = _normal(gen, K, N, std=K ** -0.5)
        # gradients of a loss averaged over the batch
        if op == "step":
            st["dY"] = _normal(gen, M, N, std=M ** -0.5)
            return st
        st["W3"] = _normal(gen, N, K, std=N ** -0.5)
        st["dZ"] = _normal(gen, M, K, std=M ** -0.5)
        # what the forward pass kept (unit variance, as A W1 and A W2 have)
        st["codes"], st["scales"] = _checkpoint(torch.randn(M, N, generator=gen, device="cuda"),
                                                torch.randn(M, N, generator=gen, device="cuda"))
        return st
    st["A"] = _activations(gen, M, K)
    if op == "down":
        st["W8"], st["s"] = _weight8(gen, K, N)
    else:
        st["W1_8"], st["s1"] = _weight8(gen, K, N)
        st["W2_8"], st["s2"] = _weight8(gen, K, N)
    if op == "mlp":
        st["W3_8"], st["s3"] = _weight8(gen, N, K)
    if own:
        # weights are laid out once, when they are loaded; the workspace is kept
        # between calls
        import swiglu_gated_mlp_amd as sw
        st["workspace"] = sw.Workspace("cuda")
        if op == "down":
            st["Wg"] = sw.swiglu_gemm_pack_weight_int8(st["W8"])
        else:
            st["Wp"] = sw.swiglu_pack_weights_int8(st["W1_8"], st["W2_8"])
        if op == "mlp":
            st["W3g"] = sw.swiglu_gemm_pack_weight_int8(st["W3_8"])
    return st


def _run_own(st):
    import swiglu_gated_mlp_amd as sw
    op = st["case"]["op"]
    if op == "mlp":
        Y, Z = sw.swiglu_mlp_packed_int8(st["A"], st["Wp"], st["s1"], st["s2"], st["W3g"], st["s3"],
                                         workspace=st["workspace"])
        return {"Y": Y, "Z": Z}
    if op == "step":
        Y, codes, scales = sw.swiglu_train_forward_int8(st["A"], st["W1"], st["W2"])
        dA, dW1, dW2 = sw.swiglu_train_backward_int8(st["dY"], st["A"], st["W1"], st["W2"], codes, scales)
        return {"Y": Y, "dA": dA, "dW1": dW1, "dW2": dW2}
    if op == "block":
        dA, dW1, dW2, dW3 = sw.swiglu_mlp_train_backward_int8(st["dZ"], st["A"], st["W1"], st["W2"], st["W3"],
                                                              st["codes"], st["scales"])
        return {"dA": dA, "dW1": dW1, "dW2": dW2, "dW3": dW3}
    A8, sa = sw.swiglu_quantize_rows_int8(st["A"])
    if op == "down":
        return {"C": sw.swiglu_gemm_packed_int8(A8, sa, st["Wg"], st["s"], workspace=st["workspace"])}
    return {"Y": sw.swiglu_fused_packed_int8(A8, sa, st["Wp"], st["s1"], st["s2"], workspace=st["workspace"])}


def _rows8(a):
    """Rows as whole numbers in -127 .. 127, and their scales."""
    top = a.abs().amax(1, keepdim=True).clamp_min(_TINY)
    return torch.round(a * (127.0 / top)), top / 127.0


def _scaled(q, sa, W8, s):
    return (q @ W8.float()) * s * sa


def _kept(codes, scales, N):
    """Gate and Up of a checkpoint, in fp32."""
    x = codes.float() * scales.float().permute(1, 0, 2)[..., None]
    M = codes.shape[0]
    x = x.permute(2, 0, 1, 3).reshape(2, M, -1)
    return x[0, :, :N], x[1, :, :N]


def run(st):
    if own:
        return _run_own(st)
    op, N = st["case"]["op"], st["case"]["N"]
    a = st["A"].float()
    if op in ("product", "down", "mlp"):
        q, sa = _rows8(a)
        if op == "down":
            return {"C": _scaled(q, sa, st["W8"], st["s"]).to(_BF16)}
        g = _scaled(q, sa, st["W1_8"], st["s1"])
        u = _scaled(q, sa, st["W2_8"], st["s2"])
        Y = (g * torch.sigmoid(g) * u).to(_BF16)
        if op == "product":
            return {"Y": Y}
        q, sy = _rows8(Y.float())
        return {"Y": Y, "Z": _scaled(q, sy, st["W3_8"], st["s3"]).to(_BF16)}
    w1, w2 = st["W1"].float(), st["W2"].float()
    out = {}
    if op == "step":
        g, u = a @ w1, a @ w2
        out["Y"] = (g * torch.sigmoid(g) * u).to(_BF16)
        codes, scales = _checkpoint(g, u)
        dy = st["dY"].float()
    else:
        codes, scales = st["codes"], st["scales"]
        dy = st["dZ"].float() @ st["W3"].float().t()
    g, u = _kept(codes, scales, N)
    s = torch.sigmoid(g)
    h = g * s
    du = dy * h
    dg = dy * u * (s * (1.0 + g * (1.0 - s)))
    out["dA"] = (dg @ w1.t() + du @ w2.t()).to(_BF16)
    out["dW1"], out["dW2"] = (a.t() @ dg).to(_BF16), (a.t() @ du).to(_BF16)
    if op == "block":
        out["dW3"] = ((h * u).t() @ st["dZ"].float()).to(_BF16)
    return out


def work(case):
    """Each input read once, each output written once, and the products'
    multiplications and additions (int8 ones in product, down and mlp)."""
    op, M, K, N = case["op"], case["M"], case["K"], case["N"]
    if op == "product":
        return {"bytes": 2 * M * K + 2 * K * N + 8 * N + 2 * M * N, "flops": 4 * M * K * N}
    if op == "down":
        return {"bytes": 2 * M * K + K * N + 4 * N + 2 * M * N, "flops": 2 * M * K * N}
    if op == "mlp":
        return {"bytes": 4 * M * K + 3 * K * N + 8 * N + 4 * K + 2 * M * N, "flops": 6 * M * K * N}
    if op == "step":
        return {"bytes": 2 * (2 * M * K + 4 * K * N + 2 * M * N), "flops": 12 * M * K * N}
    groups = (N + 31) // 32
    return {"bytes": 2 * (3 * M * K + 6 * K * N) + M * groups * (2 * 32 + 2 * 2), "flops": 12 * M * K * N}


def _quantized64(x, dim):
    """x as its codes times their scale, one scale along dim."""
    s = torch.clamp(torch.amax(torch.abs(x), dim, keepdim=True), min=_TINY) / 127.0
    return torch.round(x / s) * s


def _checkpoint64(x):
    """Gate or Up as a checkpoint gives it back, in fp64, 32 columns at a time."""
    out = torch.empty_like(x)
    for c in range(0, x.shape[1], 32):
        part = x[:, c:c + 32]
        low = torch.amax(torch.abs(part), 1, keepdim=True) / 127.0
        near = low.to(_BF16)
        up = torch.where(near.double() < low, torch.nextafter(near, torch.full_like(near, math.inf)), near)
        s = torch.clamp(up.double(), min=2.0 ** -126)
        out[:, c:c + 32] = torch.round(part / s) * s
    return out


def exact(case, seed):
    """The operators' definition in fp64.  Y, a bf16 output, is what the block's
    second product takes."""
    st = prepare(case, seed)
    op, M, N = case["op"], case["M"], case["N"]
    A = st["A"].double()
    if op in ("product", "down", "mlp"):
        def times(X, name, s):
            return torch.matmul(_quantized64(X, 1), st[name].double() * st[s].double()[None, :])
        if op == "down":
            return {"C": times(A, "W8", "s")}
        gate, up = times(A, "W1_8", "s1"), times(A, "W2_8", "s2")
        Y = gate / (1.0 + torch.exp(-gate)) * up
        if op == "product":
            return {"Y": Y}
        return {"Y": Y, "Z": times(Y.to(_BF16).double(), "W3_8", "s3")}
    W1, W2 = st["W1"].double(), st["W2"].double()
    out = {}
    if op == "step":
        gate, up = torch.matmul(A, W1), torch.matmul(A, W2)
        out["Y"] = gate / (1.0 + torch.exp(-gate)) * up
        gate, up = _checkpoint64(gate), _checkpoint64(up)
        d = st["dY"].double()
    else:
        gate, up = torch.empty(M, N, dtype=torch.float64, device=A.device), torch.empty(M, N, dtype=torch.float64,
                                                                                       device=A.device)
        for b in range((N + 31) // 32):
            cols = min(32, N - 32 * b)
            for i, x in ((0, gate), (1, up)):
                x[:, 32 * b:32 * b + cols] = (st["codes"][:, b, i, :cols].double()
                                              * st["scales"][b, :, i].double()[:, None])
        d = torch.matmul(st["dZ"].double(), st["W3"].double().T)
    sig = 1.0 / (1.0 + torch.exp(-gate))
    d_up = d * gate * sig
    # d/dg [g sig(g)] = sig(g) + g sig(g) (1 - sig(g))
    d_gate = d * up * (sig + gate * sig * (1.0 - sig))
    out["dA"] = torch.matmul(d_gate, W1.T) + torch.matmul(d_up, W2.T)
    out["dW1"], out["dW2"] = torch.matmul(A.T, d_gate), torch.matmul(A.T, d_up)
    if op == "block":
        out["dW3"] = torch.matmul((gate * sig * up).T, st["dZ"].double())
    return out
