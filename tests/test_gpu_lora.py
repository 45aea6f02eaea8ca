"""Low-rank adapters on the GPU against their definition in fp64.

Tolerances (H = 2^-8 a rounding to bf16, F = 2^-24 one to fp32, S a sum's terms in
absolute value):
  factor      t = s (A La): (K + 2) F S from its sum and scale, 2^-17 |t| from
              being held as two bf16
  sums        G = A W + t Lb: (K + 2) F S of A W, the factor's error through |Lb|,
              (2 r + 2) F S of t Lb, and F |G| for adding the two
  Y           SiLU(G) U: |SiLU'| <= 1.1, the kernels' sigmoid is off by
              (|g| + 8) 2^-23, one rounding to bf16
"""
import pytest
import torch

import swiglu_gated_mlp_amd as sw

pytestmark = pytest.mark.gpu

H = torch.finfo(torch.bfloat16).eps / 2
F = 2.0 ** -24


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return torch.device("cuda:0")


def make_ids(kind, M, L, gen, dev):
    if kind == "runs":        # one adapter a request, its rows adjacent, some without
        per = max(1, M // 5)
        ids = (torch.arange(M) // per * 3) % (L + 1) - 1
    elif kind == "mixed":     # any order, some without
        ids = torch.randint(-1, L, (M,), generator=torch.Generator().manual_seed(M + L))
    elif kind == "none":
        ids = torch.full((M,), -1)
    elif kind == "outside":   # ids that name no adapter count as none
        ids = torch.tensor([L, -7, 2 ** 31 - 1, -2 ** 31, 0, L - 1]).repeat(M // 6 + 1)[:M]
    else:
        ids = torch.full((M,), L - 1)
    return ids.to(torch.int32).to(dev)


def case(dev, M, K, N, L, r, pairs, kind, seed=0):
    g = torch.Generator(device=dev).manual_seed(97 * seed + M + 3 * K + 7 * N + 11 * r)

    def rnd(*shape, std):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(torch.bfloat16)

    t = dict(A=rnd(M, K, std=1.0), ids=make_ids(kind, M, L, g, dev),
             scales=torch.rand(L, generator=g, device=dev) * 2 + 0.25)
    for x in pairs:
        t["W" + x] = rnd(K, N, std=K ** -0.5)
        t["La" + x] = rnd(L, K, r, std=K ** -0.5)
        t["Lb" + x] = rnd(L, r, N, std=r ** -0.5)
    return t


def gated(t, r, **kw):
    Wp = sw.swiglu_pack_weights(t["W1"], t["W2"])
    Lp = sw.swiglu_lora_pack(t["La1"], t["Lb1"], t["La2"], t["Lb2"])
    return sw.swiglu_fused_packed_lora(t["A"], Wp, Lp, t["ids"], t["scales"], t["W1"].shape[1], r, **kw)


def plain(t, r, **kw):
    Wg = sw.swiglu_gemm_pack_weight(t["W"])
    Lp = sw.swiglu_gemm_lora_pack(t["La"], t["Lb"])
    return sw.swiglu_gemm_packed_lora(t["A"], Wg, Lp, t["ids"], t["scales"], t["W"].shape[1], r, **kw)


def adapted64(t, x):
    """(A W + s (A La) Lb, the bound of the fp32 result's error), fp64."""
    a, w = t["A"].double(), t["W" + x].double()
    K, r = w.shape[0], t["La" + x].shape[2]
    out, err = a @ w, (K + 2) * F * (a.abs() @ w.abs())
    for i in range(t["La" + x].shape[0]):
        rows = torch.nonzero(t["ids"] == i).flatten()
        if rows.numel() == 0:
            continue
        la, lb, s = t["La" + x][i].double(), t["Lb" + x][i].double(), float(t["scales"][i])
        low = s * (a[rows] @ la)
        e_low = (K + 2) * F * s * (a[rows].abs() @ la.abs()) + 2.0 ** -17 * low.abs()
        out[rows] += low @ lb
        err[rows] += e_low @ lb.abs() + (2 * r + 2) * F * (low.abs() @ lb.abs())
    return out, err + F * out.abs()


def check(got, ref, bound, what):
    err = (got.double() - ref).abs()
    bad = err > bound + 1e-30
    assert not bad.any() and torch.isfinite(got).all(), "%s: %d of %d outside the bound, worst %g times it" % (
        what, int(bad.sum()), bad.numel(), float((err / (bound + 1e-30)).max()))


def check_gated(Y, t, what):
    g, eg = adapted64(t, "1")
    u, eu = adapted64(t, "2")
    h = g / (1 + torch.exp(-g))
    e = u.abs() * (1.1 * eg + h.abs() * (g.abs() + 8) * 2.0 ** -23) + (h.abs() + 1.1 * eg) * eu
    check(Y, h * u, e * (1 + H) + H * (h * u).abs(), what)


def check_plain(C, t, what):
    c, e = adapted64(t, "")
    check(C, c, e * (1 + H) + H * c.abs(), what)


# every schedule of the products: decode configurations, weight panels of one and
# two row tiles, split K, 128- and 256-row tiles, the mixed launch; ragged edges;
# ranks of one and several 16-number chunks
SIZES = [(1, 64, 128, 1, 16), (1, 896, 520, 3, 4), (1, 6400, 24640, 2, 8), (7, 72, 136, 3, 1), (16, 200, 264, 5, 17),
         (20, 6152, 12360, 4, 16), (33, 896, 1032, 40, 16), (64, 520, 2056, 64, 8), (64, 264, 16648, 9, 16),
         (70, 4096, 512, 6, 16), (100, 1000, 520, 7, 64), (128, 896, 4864, 9, 16), (130, 264, 776, 50, 40),
         (200, 512, 16648, 6, 32), (300, 520, 2000, 5, 24), (700, 328, 1160, 4, 256), (1100, 1000, 520, 3, 16),
         (1100, 136, 8200, 12, 16), (2100, 200, 4000, 3, 100)]


@pytest.mark.parametrize("kind", ["runs", "mixed"])
@pytest.mark.parametrize("M,K,N,L,r", SIZES)
def test_gated(dev, M, K, N, L, r, kind):
    t = case(dev, M, K, N, L, r, ("1", "2"), kind)
    check_gated(gated(t, r), t, "%s %s" % ((M, K, N, L, r), kind))


@pytest.mark.parametrize("kind", ["runs", "mixed"])
@pytest.mark.parametrize("M,K,N,L,r", SIZES)
def test_plain(dev, M, K, N, L, r, kind):
    t = case(dev, M, K, N, L, r, ("",), kind)
    check_plain(plain(t, r), t, "%s %s" % ((M, K, N, L, r), kind))


@pytest.mark.parametrize("kind", ["runs", "mixed", "none"])
@pytest.mark.parametrize("M,K,N,r", [(66, 2056, 264, 16), (130, 2048, 264, 40), (256, 1096, 1032, 8),
                                     (257, 4864, 520, 64), (600, 4096, 264, 24), (1023, 1032, 776, 16)])
def test_split_contraction(dev, M, K, N, r, kind):
    """Few output tiles: K is split, the adapters join where the sums do."""
    t = case(dev, M, K, N, 9, r, ("1", "2", ""), kind)
    check_gated(gated(t, r), t, "%s %s" % ((M, K, N, r), kind))
    check_plain(plain(t, r), t, "%s %s" % ((M, K, N, r), kind))


@pytest.mark.parametrize("kind", ["none", "outside", "same"])
@pytest.mark.parametrize("M,K,N,L,r", [(5, 200, 264, 4, 16), (70, 4096, 512, 3, 16), (100, 72, 136, 4, 40),
                                       (600, 264, 1032, 4, 16)])
def test_id_patterns(dev, M, K, N, L, r, kind):
    t = case(dev, M, K, N, L, r, ("1", "2", ""), kind)
    Y, C = gated(t, r), plain(t, r)
    check_gated(Y, t, kind)
    check_plain(C, t, kind)
    if kind == "none":   # nothing to add: the plain products, bit for bit
        assert torch.equal(Y, sw.swiglu_fused_packed(t["A"], sw.swiglu_pack_weights(t["W1"], t["W2"]), N))
        assert torch.equal(C, sw.swiglu_gemm_packed(t["A"], sw.swiglu_gemm_pack_weight(t["W"]), N))


@pytest.mark.parametrize("M,K,N", [(24, 200, 264), (70, 4096, 512), (100, 264, 520), (300, 136, 776)])
def test_rows_are_independent(dev, M, K, N):
    """A permuted batch gives the permuted result bit for bit; an infinite row and
    an adapter of NaN and infinities change their own rows only."""
    L, r = 5, 16
    t = case(dev, M, K, N, L, r, ("1", "2", ""), "mixed")
    Y, C = gated(t, r), plain(t, r)
    perm = torch.randperm(M, generator=torch.Generator().manual_seed(1)).to(dev)
    p = dict(t, A=t["A"][perm].contiguous(), ids=t["ids"][perm].contiguous())
    assert torch.equal(gated(p, r), Y[perm]) and torch.equal(plain(p, r), C[perm])
    b = {k: v.clone() for k, v in t.items()}
    for x in ("1", "2", ""):
        b["Lb" + x][2, 3, ::5] = float("nan")
        b["Lb" + x][2, 1, 1::5] = float("inf")
        b["La" + x][2, 7, 2] = float("-inf")
    b["A"][M // 2, 5] = float("inf")
    b["A"][M // 3, 8] = float("nan")
    hurt = (t["ids"] == 2)
    hurt[M // 2] = hurt[M // 3] = True
    assert 0 < int(hurt.sum()) < M
    Yb, Cb = gated(b, r), plain(b, r)
    assert torch.equal(Yb[~hurt], Y[~hurt]) and torch.equal(Cb[~hurt], C[~hurt])
    own = (t["ids"] == 2)
    assert not torch.isfinite(Cb[own][:, ::5]).any()
    assert not torch.isfinite(Cb[M // 3]).any()


@pytest.mark.parametrize("M,K,N,r", [(700, 200, 776, 24), (2100, 72, 520, 40), (600, 2048, 520, 40)])
def test_neighbours_adapters_leave_a_row_as_it_is(dev, M, K, N, r):
    """Long batches: a row of adapter 0 gets the same bits beside rows of one, of
    three or of many other adapters, and beside adapters with NaN or infinities."""
    L = 12
    t = case(dev, M, K, N, L, r, ("1", "2", ""), "mixed")
    own = torch.arange(M, device=dev) % 5 < 2
    rest = torch.randint(1, L, (M,), generator=torch.Generator().manual_seed(2)).to(dev)
    out = []
    for others in (0, -1, 1, 1 + rest % 3, rest):
        ids = torch.where(own, torch.zeros_like(rest), torch.as_tensor(others, device=dev)).int()
        b = dict(t, ids=ids)
        Y, C = gated(b, r), plain(b, r)
        check_gated(Y, b, r"%s" % M)
        check_plain(C, b, "%s" % M)
        out.append((Y[own], C[own]))
        for x in ("1", "2", ""):
            b["Lb" + x] = t["Lb" + x].clone()
            b["Lb" + x][1:, r - 1, N - 1] = float("nan")
            b["Lb" + x][1:, 0, 1] = float("inf")
        out.append((gated(b, r)[own], plain(b, r)[own]))
    for y, c in out[1:]:
        assert torch.equal(y, out[0][0]) and torch.equal(c, out[0][1])


def fenced(t, fill):
    n, pad = t.numel(), 4096
    buf = torch.full((n + 2 * pad,), fill, dtype=t.dtype, device=t.device)
    v = buf[pad:pad + n].view(t.shape)
    v.copy_(t)
    return buf, v


@pytest.mark.parametrize("M,K,N,r", [(1, 72, 136, 4), (33, 136, 264, 17), (130, 264, 776, 16), (600, 72, 1160, 40)])
def test_nothing_outside_is_read_or_written(dev, M, K, N, r):
    """Inputs between NaNs, outputs between marks, a workspace of NaNs."""
    t = case(dev, M, K, N, 3, r, ("1", "2", ""), "mixed")
    f = {k: (fenced(v, float("nan"))[1] if v.dtype == torch.bfloat16 else v) for k, v in t.items()}
    f["ids"] = fenced(t["ids"], 0)[1]
    for fn, want, sizer in ((gated, gated(t, r), sw.swiglu_lora_workspace_bytes),
                            (plain, plain(t, r), sw.swiglu_gemm_lora_workspace_bytes)):
        need = sizer(M, K, N, r)
        ws = torch.full(((need + 3) // 4,), float("nan"), device=dev).view(torch.uint8)
        buf, out = fenced(torch.zeros_like(want), 7.0)
        fn(f, r, workspace=ws, **({"Y": out} if fn is gated else {"C": out}))
        assert torch.equal(out, want)
        assert (torch.cat((buf[:4096], buf[-4096:])) == 7.0).all()


def test_empty_batch_streams_and_graph(dev):
    M, K, N, L, r = 40, 264, 520, 6, 16
    t = case(dev, M, K, N, L, r, ("1", "2", ""), "mixed")
    assert gated(dict(t, A=t["A"][:0], ids=t["ids"][:0]), r).shape == (0, N)
    Wp, Lp = sw.swiglu_pack_weights(t["W1"], t["W2"]), sw.swiglu_lora_pack(t["La1"], t["Lb1"], t["La2"], t["Lb2"])
    Wg, Lq = sw.swiglu_gemm_pack_weight(t["W"]), sw.swiglu_gemm_lora_pack(t["La"], t["Lb"])

    def run(A, ids, **kw):
        return (sw.swiglu_fused_packed_lora(A, Wp, Lp, ids, t["scales"], N, r, **kw),
                sw.swiglu_gemm_packed_lora(A, Wg, Lq, ids, t["scales"], N, r, **kw))

    want = run(t["A"], t["ids"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = run(t["A"], t["ids"], stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    A, ids = t["A"].clone(), t["ids"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run(A, ids)
    for seed in (1, 2, 3):
        fresh = case(dev, M, K, N, L, r, (), ("runs", "mixed", "none")[seed - 1], seed=seed)
        A.copy_(fresh["A"])
        ids.copy_(fresh["ids"])
        want = run(fresh["A"], fresh["ids"])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), seed
