"""Training and adapter operators of the gated MLP block, as they are measured.

Every case is one pass through one operator on bf16 tensors on the GPU:

  forward         Y = SiLU(G) * U with G = A W1, U = A W2; G and U are kept for
                  the backward pass and returned too
  backward        dA, dW1, dW2 from dY, either with the kept G and U or (keep
                  false) with G and U computed again from A, W1, W2
  block           the backward pass of the whole block Z = Y W3, from dZ: dA,
                  dW1, dW2, dW3
  adapters        Y = SiLU(G) * U with G = A W1 + s_i (A La1_i) Lb1_i and U alike,
                  i = ids[m] the low-rank adapter of row m (-1: none)
  adapters_down   C = A W + s_i (A La_i) Lb_i, the same beside one projection

``own`` False computes them in fp32 with elementary torch operations, ``own``
True through swiglu_gated_mlp_amd.  The widths are the repository's workloads
(K x N of the gate/up projections 896 x 4864, 3584 x 18944 and 8192 x 29568) and
odd ones between them.
"""
from __future__ import annotations

import math

import torch

own = False

_BF16 = torch.bfloat16


def listed():
    return [
        # keeping Gate and Up for the backward pass: one short sequence at the
        # smallest width (latency), and a training batch at the 7B width
        dict(name="forward-0.5b-m64", op="forward", M=64, K=896, N=4864),
        dict(name="forward-7b-m4096", op="forward", M=4096, K=3584, N=18944),
        # gradients with Gate and Up kept: a batch at the smallest width, the
        # largest batch at the 7B width, and recomputation (activation
        # checkpointing) on a ragged batch at a width that no tile divides
        dict(name="backward-0.5b-m4096", op="backward", M=4096, K=896, N=4864, keep=True),
        dict(name="backward-7b-m8192", op="backward", M=8192, K=3584, N=18944, keep=True),
        dict(name="recompute-odd-m1003", op="backward", M=1003, K=1416, N=5896, keep=False),
        # the whole block's gradients: a last, short micro-batch, and a
        # 2048-token one at the 7B width
        dict(name="block-0.5b-m333", op="block", M=333, K=896, N=4864),
        dict(name="block-7b-m2048", op="block", M=2048, K=3584, N=18944),
        # serving: one request's next token; a decode batch in which nearly
        # every request has its own adapter; a prefill batch of a few requests
        dict(name="adapters-7b-m1", op="adapters", M=1, K=3584, N=18944, L=16, r=16, requests=1),
        dict(name="adapters-7b-m32", op="adapters", M=32, K=3584, N=18944, L=48, r=16, requests=32),
        dict(name="adapters-7b-m2100", op="adapters", M=2100, K=3584, N=18944, L=8, r=32, requests=6),
        # the down projection of the same block: a decode batch, and a prefill
        # at the smallest width
        dict(name="adapters-down-7b-m16", op="adapters_down", M=16, K=18944, N=3584, L=32, r=16, requests=16),
        dict(name="adapters-down-0.5b-m2000", op="adapters_down", M=2000, K=4864, N=896, L=8, r=64, requests=5),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the listed ones' ranges: widths from 128 x 256 to the 72B one,
    1 to 8192 rows, ranks 4 to 64, no dearer than the 8192-row backward."""
    op = rng.choice(["forward", "backward", "backward", "block", "adapters", "adapters", "adapters_down"])
    limit = 8192 * 3584 * 18944
    while True:
        M = _log_int(rng, 1, 8192)
        K = 8 * _log_int(rng, 16, 1024)
        N = 8 * _log_int(rng, 32, 3696)
        if op == "adapters_down":
            K, N = N, K
        cost = M * K * N * {"forward": 0.5, "backward": 1.5, "block": 1.5}.get(op, 0.75)
        # tiny widths with a handful of rows would only time the launch
        if cost <= limit and K * N >= 1 << 18:
            break
    case = dict(op=op, M=M, K=K, N=N)
    if op == "backward":
        case["keep"] = rng.random() < 0.6
    if op.startswith("adapters"):
        case["r"] = rng.choice([4, 8, 16, 24, 32, 64])
        case["L"] = rng.choice([1, 3, 8, 16, 32])
        case["requests"] = min(M, _log_int(rng, 1, 64))
    return case


def _normal(gen, *shape, std=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(_BF16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op, M, K, N = case["op"], case["M"], case["K"], case["N"]
    st = {"case": dict(case)}
    st["A"] = _normal(gen, M, K)
    if op in ("forward", "backward", "block"):
        st["W1"] = _normal(gen, K, N, std=K ** -0.5)
        st["W2"] = _normal(gen, K, N, std=K ** -0.5)
        # gradients of a loss averaged over the batch
        if op == "backward":
            st["dY"] = _normal(gen, M, N, std=M ** -0.5)
        if op == "block":
            st["W3"] = _normal(gen, N, K, std=N ** -0.5)
            st["dZ"] = _normal(gen, M, K, std=M ** -0.5)
        if op == "block" or case.get("keep"):
            # what the forward pass kept (unit variance, as A W1 and A W2 have)
            st["G"] = _normal(gen, M, N)
            st["U"] = _normal(gen, M, N)
        if op == "block":
            g = st["G"].float()
            st["Y"] = (g * torch.sigmoid(g) * st["U"].float()).to(_BF16)
        return st
    L, r = case["L"], case["r"]
    names = ("1", "2") if op == "adapters" else ("",)
    for x in names:
        st["W" + x] = _normal(gen, K, N, std=K ** -0.5)
        st["La" + x] = _normal(gen, L, K, r, std=K ** -0.5)
        st["Lb" + x] = _normal(gen, L, r, N, std=0.5 * r ** -0.5)
    st["scales"] = torch.rand(L, generator=gen, device="cuda") * 1.5 + 0.5
    # one adapter a request (one request in eight has none); a request's rows
    # are adjacent, as a scheduler lays a batch out
    cpu = torch.Generator().manual_seed(int(seed) + 1)
    R = case["requests"]
    cuts = torch.sort(torch.randperm(M - 1, generator=cpu)[:R - 1] + 1).values.tolist() if R > 1 else []
    edges = [0] + cuts + [M]
    ids = torch.empty(M, dtype=torch.int32)
    order = torch.randperm(L, generator=cpu).tolist()
    for q in range(R):
        ids[edges[q]:edges[q + 1]] = -1 if q % 8 == 7 else order[q % L]
    st["ids"] = ids.cuda()
    if own:
        # weights and adapters are laid out once, when they are loaded; the
        # workspace is kept between calls
        import swiglu_gated_mlp_amd as sw
        st["workspace"] = sw.Workspace("cuda")
        if op == "adapters":
            st["Wp"] = sw.swiglu_pack_weights(st["W1"], st["W2"])
            st["Lp"] = sw.swiglu_lora_pack(st["La1"], st["Lb1"], st["La2"], st["Lb2"])
        else:
            st["Wg"] = sw.swiglu_gemm_pack_weight(st["W"])
            st["Lp"] = sw.swiglu_gemm_lora_pack(st["La"], st["Lb"])
    return st


def _run_own(st):
    import swiglu_gated_mlp_amd as sw
    op = st["case"]["op"]
    if op == "forward":
        Y, G, U = sw.swiglu_train_forward(st["A"], st["W1"], st["W2"])
        return {"Y": Y, "G": G, "U": U}
    if op == "backward":
        dA, dW1, dW2 = sw.swiglu_train_backward(st["dY"], st["A"], st["W1"], st["W2"], st.get("G"), st.get("U"))
        return {"dA": dA, "dW1": dW1, "dW2": dW2}
    if op == "block":
        dA, dW1, dW2, dW3 = sw.swiglu_mlp_train_backward(st["dZ"], st["A"], st["W1"], st["W2"], st["W3"], st["G"],
                                                         st["U"], st["Y"])
        return {"dA": dA, "dW1": dW1, "dW2": dW2, "dW3": dW3}
    N, r = st["case"]["N"], st["case"]["r"]
    if op == "adapters":
        return {"Y": sw.swiglu_fused_packed_lora(st["A"], st["Wp"], st["Lp"], st["ids"], st["scales"], N, r,
                                                 workspace=st["workspace"])}
    return {"C": sw.swiglu_gemm_packed_lora(st["A"], st["Wg"], st["Lp"], st["ids"], st["scales"], N, r,
                                            workspace=st["workspace"])}


def _adapted(a, W, La, Lb, ids, scales):
    """A W + s_i (A La_i) Lb_i in fp32: every row times every adapter's first
    factor, the other adapters' columns set to zero, times the second factors."""
    L, K, r = La.shape
    t = a @ La.float().permute(1, 0, 2).reshape(K, L * r)
    mine = (ids[:, None] == torch.arange(L, device=ids.device)[None, :]).float() * scales[None, :]
    t = (t.view(-1, L, r) * mine[:, :, None]).reshape(-1, L * r)
    return a @ W.float() + t @ Lb.float().reshape(L * r, -1)


def run(st):
    if own:
        return _run_own(st)
    op = st["case"]["op"]
    a = st["A"].float()
    if op.startswith("adapters"):
        ids, sc = st["ids"], st["scales"]
        if op == "adapters_down":
            return {"C": _adapted(a, st["W"], st["La"], st["Lb"], ids, sc).to(_BF16)}
        g = _adapted(a, st["W1"], st["La1"], st["Lb1"], ids, sc)
        u = _adapted(a, st["W2"], st["La2"], st["Lb2"], ids, sc)
        return {"Y": (g * torch.sigmoid(g) * u).to(_BF16)}
    w1, w2 = st["W1"].float(), st["W2"].float()
    if op == "forward":
        g, u = a @ w1, a @ w2
        return {"Y": (g * torch.sigmoid(g) * u).to(_BF16), "G": g.to(_BF16), "U": u.to(_BF16)}
    if "G" in st:
        g, u = st["G"].float(), st["U"].float()
    else:
        g, u = a @ w1, a @ w2
    dy = st["dZ"].float() @ st["W3"].float().t() if op == "block" else st["dY"].float()
    s = torch.sigmoid(g)
    h = g * s
    du = dy * h
    dg = dy * u * (s * (1.0 + g * (1.0 - s)))
    out = {"dA": (dg @ w1.t() + du @ w2.t()).to(_BF16), "dW1": (a.t() @ dg).to(_BF16), "dW2": (a.t() @ du).to(_BF16)}
    if op == "block":
        out["dW3"] = (st["Y"].float().t() @ st["dZ"].float()).to(_BF16)
    return out


def work(case):
    """Each input read once, each output written once (2 bytes an element), and
    the products' multiplications and additions."""
    op, M, K, N = case["op"], case["M"], case["K"], case["N"]
    if op == "forward":
        return {"bytes": 2 * (M * K + 2 * K * N + 3 * M * N), "flops": 4 * M * K * N}
    if op == "backward":
        keep = bool(case["keep"])
        return {"bytes": 2 * (2 * M * K + 4 * K * N + (3 if keep else 1) * M * N),
                "flops": (8 if keep else 12) * M * K * N}
    if op == "block":
        return {"bytes": 2 * (3 * M * K + 6 * K * N + 3 * M * N), "flops": 12 * M * K * N}
    pairs = 2 if op == "adapters" else 1
    L, r, R = case["L"], case["r"], case["requests"]
    used = min(L, R - R // 8) if R > 1 else 1
    return {"bytes": 2 * (M * K + pairs * K * N + M * N + pairs * used * r * (K + N)) + 4 * M + 4 * used,
            "flops": pairs * (2 * M * K * N + 2 * M * r * (K + N))}


def exact(case, seed):
    """The operators' definition in fp64, adapters taken one at a time."""
    st = prepare(case, seed)
    d = {k: v.double() for k, v in st.items() if isinstance(v, torch.Tensor) and v.dtype == _BF16
         and k in ("A", "W", "W1", "W2", "W3", "dY", "dZ", "G", "U", "Y", "La", "Lb", "La1", "Lb1", "La2", "Lb2")}
    op = case["op"]
    if op.startswith("adapters"):
        def projected(x):
            out = torch.matmul(d["A"], d["W" + x])
            for i in range(case["L"]):
                rows = torch.nonzero(st["ids"] == i).flatten()
                if rows.numel():
                    low = torch.matmul(d["A"][rows], d["La" + x][i])
                    out[rows] += float(st["scales"][i]) * torch.matmul(low, d["Lb" + x][i])
            return out
        if op == "adapters_down":
            return {"C": projected("")}
        gate, up = projected("1"), projected("2")
        return {"Y": gate / (1.0 + torch.exp(-gate)) * up}
    if "G" in d:
        gate, up = d["G"], d["U"]
    else:
        gate, up = torch.matmul(d["A"], d["W1"]), torch.matmul(d["A"], d["W2"])
    sig = 1.0 / (1.0 + torch.exp(-gate))
    if op == "forward":
        return {"Y": gate * sig * up, "G": gate, "U": up}
    dy = torch.matmul(d["dZ"], d["W3"].T) if op == "block" else d["dY"]
    d_up = dy * gate * sig
    # d/dg [g sig(g)] = sig(g) + g sig(g) (1 - sig(g))
    d_gate = dy * up * (sig + gate * sig * (1.0 - sig))
    out = {"dA": torch.matmul(d_gate, d["W1"].T) + torch.matmul(d_up, d["W2"].T),
           "dW1": torch.matmul(d["A"].T, d_gate), "dW2": torch.matmul(d["A"].T, d_up)}
    if op == "block":
        out["dW3"] = torch.matmul(d["Y"].T, d["dZ"])
    return out
