"""The int8 products on the GPU against their definition, whole numbers exactly
(fp64 holds every sum of codes below 2^53) and the rest in fp64.

Tolerances.  A rounding to fp32 is off by at most 2^-24 of the value, one to bf16
by 2^-8.
  codes, scales   equal to the definition's own fp32 steps
  G, U, C         the sum's rounding to fp32 and two products: 3 roundings to fp32
  SiLU            the kernels' sigmoid: relative error (|g| + 8) 2^-23 (the rounding
                  of g log2 e scales with |g|; a few ulp for the rest); |SiLU'| <= 1.1
  C, Y, Z         one rounding to bf16 besides
"""
import pytest
import torch

import swiglu_gated_mlp_amd as sw

pytestmark = pytest.mark.gpu

H = torch.finfo(torch.bfloat16).eps / 2   # 2^-8
F = 2.0 ** -24
TINY = 2.0 ** -96


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return torch.device("cuda:0")


def quantized(x, dim):
    """The definition's steps, in fp32: codes along dim, scales.  (Tensors on both
    sides of a division: torch multiplies by a number's reciprocal instead.)"""
    x = x.float()
    c = torch.full((), 127.0, device=x.device).expand_as(x.amax(dim, keepdim=True)).contiguous()
    top = x.abs().amax(dim, keepdim=True)
    good = torch.isfinite(top)
    t = top.clamp_min(TINY)
    q = torch.where(good, torch.round(x * (c / t)), torch.zeros_like(x))
    return q.nan_to_num(0.0).to(torch.int8), torch.where(good, t / c, torch.full_like(t, float("nan"))).squeeze(dim)


def same(a, b):
    return torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(0.0), b.nan_to_num(0.0))


def activations(dev, M, K, seed):
    g = torch.Generator(device=dev).manual_seed(seed)
    a = torch.randn(M, K, generator=g, device=dev) * torch.exp(torch.randn(M, 1, generator=g, device=dev))
    return a.to(torch.bfloat16)


def codes(dev, R, C, seed):
    g = torch.Generator(device=dev).manual_seed(seed)
    return torch.randint(-127, 128, (R, C), generator=g, device=dev, dtype=torch.int8)


def scales(dev, n, seed, unit):
    g = torch.Generator(device=dev).manual_seed(seed)
    return (torch.rand(n, generator=g, device=dev) + 0.5) * unit


def sums(A, W):
    return torch.matmul(A.double(), W.double())


def check(got, ref, bound, what):
    assert torch.isfinite(got).all(), what
    err = (got.double() - ref).abs()
    bad = err > bound + 1e-38
    assert not bad.any(), "%s: %d of %d outside the bound, worst %g times it" % (
        what, int(bad.sum()), bad.numel(), float((err / (bound + 1e-38)).max()))


def check_gemm(C, A, sa, W, s, what):
    ref = sums(A, W) * s.double() * sa.double()[:, None]
    check(C, ref, ref.abs() * (H * (1 + 4 * F) + 3.01 * F), what)


def check_fused(Y, A, sa, W1, s1, W2, s2, what):
    g, u = (sums(A, W) * s.double() * sa.double()[:, None] for W, s in ((W1, s1), (W2, s2)))
    h = g / (1.0 + torch.exp(-g))
    ref = h * u
    e = 1.1 * 3.01 * F * g.abs() * u.abs() + ref.abs() * (3.01 * F + (g.abs() + 8) * 2 * F + 2 * F)
    check(Y, ref, e + (ref.abs() + e) * H, what)


# units that give G and U of about 1: sums of K products of codes of about 73 each
def pair(dev, M, K, N, seed):
    unit = (73.0 * 73.0 * K ** 0.5) ** -0.5
    return (codes(dev, M, K, seed), scales(dev, M, seed + 1, unit), codes(dev, K, N, seed + 2),
            scales(dev, N, seed + 3, unit), codes(dev, K, N, seed + 4), scales(dev, N, seed + 5, unit))


@pytest.mark.parametrize("M,K", [(1, 8), (3, 16), (5, 1000), (4, 1024), (2, 1032), (77, 4096), (3, 4104), (9, 8192),
                                 (2, 8200), (33, 18944), (2, 32776), (2, 131056)])
def test_rows(dev, M, K):
    A = activations(dev, M, K, M + K)
    Q, s = sw.swiglu_quantize_rows_int8(A)
    q, t = quantized(A, 1)
    assert torch.equal(Q, q) and torch.equal(s, t)


@pytest.mark.parametrize("K,N", [(8, 8), (40, 72), (1000, 136), (3584, 896)])
def test_columns(dev, K, N):
    W = activations(dev, N, K, K + N).t().contiguous()
    Q, s = sw.swiglu_quantize_columns_int8(W)
    q, t = quantized(W, 0)
    assert torch.equal(Q, q) and torch.equal(s, t)


def special_rows(dev, K):
    big = torch.finfo(torch.bfloat16).max
    A = activations(dev, 16, K, 5)
    A[0] = 0
    A[1] *= 2.0 ** -110           # below the least maximum
    A[2, K // 2] = float("inf")
    A[3, 0] = float("nan")
    A[4, K - 1] = -float("inf")
    A[5, 1] = big
    A[6] = -big
    A[7] = 127 * 2.0 ** -7        # every value on a tie's border
    A[7, 1:] = torch.arange(K - 1, device=dev).remainder(127).add(0.5).mul(2.0 ** -7).to(torch.bfloat16)
    A[8] = 2.0 ** -130            # subnormal
    return A


@pytest.mark.parametrize("K", [64, 1008, 4112])
def test_special_values(dev, K):
    A = special_rows(dev, K)
    for X, dim, call in ((A, 1, sw.swiglu_quantize_rows_int8), (A.t().contiguous(), 0, sw.swiglu_quantize_columns_int8)):
        Q, s = call(X)
        q, t = quantized(X, dim)
        assert torch.equal(Q, q) and same(s, t)
        assert s.isnan().nonzero().flatten().tolist() == [2, 3, 4]


def test_a_bad_row_or_column_stays_its_own(dev):
    K, N = 64, 80
    A = special_rows(dev, K)
    clean = A.clone()
    clean[2:5] = 1.0
    W = [activations(dev, K, N, 7 + i) for i in range(3)]
    W8 = [sw.swiglu_quantize_columns_int8(w) for w in W]
    bad = W8[0][1].clone()
    bad[11] = float("nan")
    Wp, Wg = sw.swiglu_pack_weights_int8(W8[0][0], W8[1][0]), sw.swiglu_gemm_pack_weight_int8(W8[2][0])

    def both(X, s1):
        Q, s = sw.swiglu_quantize_rows_int8(X)
        return sw.swiglu_fused_packed_int8(Q, s, Wp, s1, W8[1][1]), sw.swiglu_gemm_packed_int8(Q, s, Wg, W8[2][1])

    for got, want in zip(both(A, W8[0][1]), both(clean, W8[0][1])):
        assert got[2:5].isnan().all()
        for r in (0, 1, *range(5, 16)):
            assert same(got[r], want[r])
    got, want = both(clean, bad)[0], both(clean, W8[0][1])[0]
    assert got[:, 11].isnan().all()
    keep = torch.arange(N, device=dev) != 11
    assert same(got[:, keep], want[:, keep])


def test_pack_layout(dev):
    for K, N in [(128, 128), (144, 136), (896, 520), (16, 8)]:
        W1, W2 = codes(dev, K, N, K), codes(dev, K, N, N)
        KB = (K + 127) // 128
        for single in (False, True):
            P = (sw.swiglu_gemm_pack_weight_int8(W1) if single else sw.swiglu_pack_weights_int8(W1, W2)).cpu()
            cols = 256 if single else 128
            tiles = (N + cols - 1) // cols
            assert P.numel() == tiles * KB * 32768
            # [tile][block][group g][half h][lane l][e] -> [column][k]
            P = P.view(tiles, KB, 16, 2, 4, 16, 16).permute(0, 2, 5, 1, 3, 4, 6).reshape(tiles, 256, KB * 128)
            for W, rows in ((W1, slice(0, cols)),) if single else ((W1, slice(0, 128)), (W2, slice(128, 256))):
                got = P[:, rows].reshape(tiles * cols, KB * 128)
                want = torch.zeros_like(got)
                want[:N, :K] = W.t().cpu()
                assert torch.equal(got, want)


# every kernel: one to 64 rows (each count of 16-row tiles, wide and narrow groups), few rows (each tile, whole and in
# parts), many rows (panels, persistent 256-row tiles with and without a tail); ragged K and N
SHAPES = [(1, 16, 8), (1, 896, 4864), (4, 1040, 520), (5, 2064, 520), (7, 144, 136), (8, 896, 512), (9, 912, 520),
          (1, 1040, 25000), (16, 1040, 25000), (16, 13312, 264), (17, 1024, 1040), (30, 8192, 24584), (32, 2064, 19000),
          (12, 2064, 65544), (31, 2064, 65544), (33, 896, 4864), (34, 128, 64), (48, 912, 1032), (64, 4880, 904),
          (37, 1760, 64), (48, 13312, 16392), (64, 912, 4872), (50, 2048, 18944), (65, 896, 4864), (65, 272, 72),
          (66, 9120, 5872), (70, 400, 8312), (70, 7216, 8280), (70, 7504, 16624), (71, 2960, 2712), (74, 656, 64),
          (76, 576, 18744), (69, 7664, 5872), (82, 416, 16768), (100, 4096, 18952), (128, 3584, 8200), (129, 912, 1032),
          (149, 1744, 23056), (180, 1040, 19000), (200, 8192, 29568), (220, 400, 19688), (256, 896, 4864),
          (300, 4112, 1032), (300, 9008, 20008), (414, 16064, 1368), (400, 912, 33000), (512, 896, 4864),
          (513, 1040, 904), (655, 144, 19880), (656, 2544, 10192), (972, 144, 29584), (1100, 2000, 4872),
          (1159, 1600, 10816), (1196, 2576, 12472), (1300, 3600, 18952), (1816, 2576, 264), (1800, 3600, 18952),
          (2100, 1024, 9000), (2706, 7216, 72), (2729, 14912, 400), (100, 16000, 520), (200, 16000, 1000),
          (1030, 4112, 1000), (33, 18416, 1056), (174, 16, 5160), (33, 1232, 14568), (259, 6368, 56), (36, 7408, 4128),
          (65, 23584, 1040), (73, 13408, 1624), (334, 10736, 1432), (70, 11952, 4144), (1513, 15248, 256),
          (69, 19024, 6264), (70, 2576, 12960), (35, 5984, 8320), (66, 10032, 4360), (1359, 14736, 488),
          (65, 15200, 8368), (4197, 9584, 88), (70, 20016, 4112), (602, 16, 6464), (2067, 22896, 200), (4169, 9056, 440),
          (65, 12736, 16488), (19, 14832, 4240), (20, 16, 17144), (21, 9504, 8272), (22, 656, 22720), (26, 1200, 13120),
          (30, 16, 13512), (32, 9440, 4096), (529, 4592, 440), (28, 24352, 848), (8, 16384, 1024), (1, 16384, 5120),
          (25, 5712, 4224), (26, 400, 17032), (31, 416, 12664), (579, 16960, 864)]


@pytest.mark.parametrize("M,K,N", SHAPES)
def test_products(dev, M, K, N):
    A, sa, W1, s1, W2, s2 = pair(dev, M, K, N, M + K + N)
    Y = sw.swiglu_fused_packed_int8(A, sa, sw.swiglu_pack_weights_int8(W1, W2), s1, s2)
    check_fused(Y, A, sa, W1, s1, W2, s2, "fused")
    C = sw.swiglu_gemm_packed_int8(A, sa, sw.swiglu_gemm_pack_weight_int8(W1), s1)
    check_gemm(C, A, sa, W1, s1, "gemm")


def test_every_kernel_is_met(dev):
    """The shapes above, as they are planned on this device."""
    met = set()
    for gemm in (False, True):
        for shape in SHAPES:
            p = sw.swiglu_probe_int8_plan(gemm, *shape)
            tile = (gemm, p["kernel"], p["rows"], p["cols"])
            met |= {tile, tile + ("parts", p["splits"] > 1), tile + ("once", p["once"])}
    for gemm in (False, True):
        for rows, cols in ((32, 96), (32, 128), (64, 96), (64, 128), (128, 128), (128, 256)) + (
                () if gemm else ((32, 160), (64, 160), (128, 192))):
            for what in ("parts", "once"):
                for yes in (False, True):
                    assert (gemm, "narrow", rows, cols, what, yes) in met, (gemm, rows, cols, what, yes)
        for rows in (16, 32) + ((64,) if gemm else ()):
            assert (gemm, "decode", rows, 256) in met
        assert (gemm, "stream", 256, 256) in met
    assert (False, "stream", 256, 64) in met


@pytest.mark.parametrize("M", [1, 40, 100, 300])
def test_largest_sums(dev, M):
    """Codes of -128 over the longest contraction: 2^14 * 131056 < 2^31."""
    K, N = 131056, 24
    A, W = torch.full((M, K), -128, dtype=torch.int8, device=dev), torch.full((K, N), -128, dtype=torch.int8, device=dev)
    W[:, 1::2] = 127
    sa, s = scales(dev, M, 1, 2.0 ** -15), scales(dev, N, 2, 2.0 ** -15)
    check_gemm(sw.swiglu_gemm_packed_int8(A, sa, sw.swiglu_gemm_pack_weight_int8(W), s), A, sa, W, s, "gemm")
    one = torch.ones(N, device=dev) * 2.0 ** -15
    Y = sw.swiglu_fused_packed_int8(A, sa, sw.swiglu_pack_weights_int8(W, W), s, one)
    check_fused(Y, A, sa, W, s, W, one, "fused")


def test_scales_at_any_word(dev):
    """Scales that begin at any 4 bytes."""
    for M in (5, 70, 600):
        K, N = 256, 520
        A, sa, W1, s1, W2, s2 = pair(dev, M, K, N, M)
        buf = torch.zeros(2 * N + M + 6, device=dev)
        v1, v2, va = buf[1:1 + N], buf[N + 3:2 * N + 3], buf[2 * N + 4:2 * N + 4 + M]
        v1.copy_(s1), v2.copy_(s2), va.copy_(sa)
        Wp, Wg = sw.swiglu_pack_weights_int8(W1, W2), sw.swiglu_gemm_pack_weight_int8(W1)
        assert torch.equal(sw.swiglu_fused_packed_int8(A, va, Wp, v1, v2), sw.swiglu_fused_packed_int8(A, sa, Wp, s1, s2))
        assert torch.equal(sw.swiglu_gemm_packed_int8(A, va, Wg, v1), sw.swiglu_gemm_packed_int8(A, sa, Wg, s1))


def block(dev, M, K, N, seed):
    A = activations(dev, M, K, seed)
    W = [activations(dev, N, K, seed + 1).t().contiguous() * K ** -0.5, activations(dev, N, K, seed + 2).t().contiguous()
         * K ** -0.5, activations(dev, K, N, seed + 3).t().contiguous() * N ** -0.5]
    W8 = [sw.swiglu_quantize_columns_int8(w) for w in W]
    Wp, W3g = sw.swiglu_pack_weights_int8(W8[0][0], W8[1][0]), sw.swiglu_gemm_pack_weight_int8(W8[2][0])
    return A, (Wp, W8[0][1], W8[1][1], W3g, W8[2][1]), W8


@pytest.mark.parametrize("M,K,N", [(1, 64, 80), (5, 896, 4864), (64, 896, 4864), (100, 1040, 2064), (333, 896, 4864),
                                   (700, 144, 1040)])
def test_block(dev, M, K, N):
    """The block is its steps, bit for bit, and the steps are their definition."""
    A, w, W8 = block(dev, M, K, N, M)
    ws = sw.Workspace(dev)
    Y, Z = sw.swiglu_mlp_packed_int8(A, *w, workspace=ws)
    Q, sa = sw.swiglu_quantize_rows_int8(A)
    Y1 = sw.swiglu_fused_packed_int8(Q, sa, w[0], w[1], w[2])
    Q3, sy = sw.swiglu_quantize_rows_int8(Y1)
    Z1 = sw.swiglu_gemm_packed_int8(Q3, sy, w[3], w[4])
    assert torch.equal(Y, Y1) and torch.equal(Z, Z1)
    check_fused(Y, Q, sa, W8[0][0], w[1], W8[1][0], w[2], "Y")
    check_gemm(Z, Q3, sy, W8[2][0], w[4], "Z")
    # again in the same workspace, and in one full of NaN
    ws.buf.fill_(0xFF)
    again = sw.swiglu_mlp_packed_int8(A, *w, workspace=ws)
    assert torch.equal(Y, again[0]) and torch.equal(Z, again[1])


def test_rows_behind_the_last_are_left(dev):
    M, K, N = 37, 144, 136
    A, sa, W1, s1, W2, s2 = pair(dev, M, K, N, 3)
    for m in (1, 37):
        Y = torch.full((m + 3, N), 7.0, dtype=torch.bfloat16, device=dev)
        sw.swiglu_fused_packed_int8(A[:m], sa[:m], sw.swiglu_pack_weights_int8(W1, W2), s1, s2, Y=Y[:m])
        C = torch.full((m + 3, N), 7.0, dtype=torch.bfloat16, device=dev)
        sw.swiglu_gemm_packed_int8(A[:m], sa[:m], sw.swiglu_gemm_pack_weight_int8(W1), s1, C=C[:m])
        assert (Y[m:] == 7).all() and (C[m:] == 7).all()
        X = activations(dev, m, K, m)
        Q, s = torch.full((m + 2, K), 5, dtype=torch.int8, device=dev), torch.full((m + 2,), 5.0, device=dev)
        sw.swiglu_quantize_rows_int8(X, Q[:m], s[:m])
        assert (Q[m:] == 5).all() and (s[m:] == 5).all()


def test_empty_batch(dev):
    A, w, _ = block(dev, 1, 64, 80, 1)
    Y, Z = sw.swiglu_mlp_packed_int8(A[:0], *w)
    assert Y.shape == (0, 80) and Z.shape == (0, 64)
    Q, s = sw.swiglu_quantize_rows_int8(A[:0])
    assert Q.shape == (0, 64) and s.shape == (0,)
    assert sw.swiglu_fused_packed_int8(Q, s, *w[:3]).shape == (0, 80)


@pytest.mark.parametrize("M", [1, 40, 100, 700])
def test_captured_and_replayed(dev, M):
    """The whole block in a graph, replayed on new inputs between eager calls."""
    A, w, _ = block(dev, M, 896, 1040, M)
    ws = sw.Workspace(dev)
    sw.swiglu_mlp_packed_int8(A, *w, workspace=ws)   # grown, and the library loaded
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    held = A.clone()
    with torch.cuda.graph(graph, stream=side):
        Y, Z = sw.swiglu_mlp_packed_int8(held, *w)
    for i in range(4):
        X = activations(dev, M, 896, 100 + i)
        held.copy_(X)
        graph.replay()
        y, z = sw.swiglu_mlp_packed_int8(X, *w, workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(Y, y) and torch.equal(Z, z)


def test_on_another_stream(dev):
    A, w, _ = block(dev, 70, 896, 1040, 2)
    want = sw.swiglu_mlp_packed_int8(A, *w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = sw.swiglu_mlp_packed_int8(A, *w, stream=s)
    q = sw.swiglu_quantize_rows_int8(A, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(q[0], sw.swiglu_quantize_rows_int8(A)[0])


def test_activations_past_2gib(dev):
    """Row chunks: the offsets of an activation pass 31 bits."""
    K, N = 131056, 24
    M = (1 << 31) // K + 300
    A, W = codes(dev, M, K, 1), codes(dev, K, N, 2)
    sa, s = scales(dev, M, 3, 2.0 ** -11), scales(dev, N, 4, 2.0 ** -11)
    C = sw.swiglu_gemm_packed_int8(A, sa, sw.swiglu_gemm_pack_weight_int8(W), s)
    Y = sw.swiglu_fused_packed_int8(A, sa, sw.swiglu_pack_weights_int8(W, W), s, s)
    for r in (slice(0, 300), slice(M // 2, M // 2 + 300), slice(M - 300, M)):
        check_gemm(C[r], A[r], sa[r], W, s, "gemm")
        check_fused(Y[r], A[r], sa[r], W, s, W, s, "fused")


@pytest.mark.parametrize("M,K,N", [(140000, 64, 16384), (1100000, 16, 2056)])
def test_outputs_past_2gib(dev, M, K, N):
    """Offsets of an output pass 31 bits; over a million rows."""
    A, sa, W1, s1, W2, s2 = pair(dev, M, K, N, 9)
    Y = sw.swiglu_fused_packed_int8(A, sa, sw.swiglu_pack_weights_int8(W1, W2), s1, s2)
    C = sw.swiglu_gemm_packed_int8(A, sa, sw.swiglu_gemm_pack_weight_int8(W1), s1)
    for r in (slice(0, 300), slice(M // 2, M // 2 + 300), slice(M - 300, M)):
        check_fused(Y[r], A[r], sa[r], W1, s1, W2, s2, "fused")
        check_gemm(C[r], A[r], sa[r], W1, s1, "gemm")


def test_quantizing_past_2gib(dev):
    """Over a million short rows, and elements past 31 bits."""
    for M, K in ((1100000, 16), (70000, 32768)):
        A = activations(dev, M, K, 1)
        Q, s = sw.swiglu_quantize_rows_int8(A)
        for r in (slice(0, 300), slice(M // 2, M // 2 + 300), slice(M - 300, M)):
            q, t = quantized(A[r], 1)
            assert torch.equal(Q[r], q) and torch.equal(s[r], t)
    Q, s = sw.swiglu_quantize_columns_int8(A)
    for c in (slice(0, 64), slice(K // 2, K // 2 + 64), slice(K - 64, K)):
        q, t = quantized(A[:, c], 0)
        assert torch.equal(Q[:, c], q) and torch.equal(s[c], t)
