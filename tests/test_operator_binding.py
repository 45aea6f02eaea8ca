"""The Python side of the training and adapter operators without a GPU: the calls run
on CPU tensors, and a stand-in for the library records what reaches its entry points
(its host functions, the workspace sizes, are the library's own)."""
import threading

import pytest
import torch

import swiglu_gated_mlp_amd as sw

BF = dict(dtype=torch.bfloat16)


class StandIn:
    """The library with its launching entry points replaced: each call is recorded and
    handed to `launch(name, args)`."""

    def __init__(self, real, launch=None):
        self.real, self.launch, self.calls = real, launch, []

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return getattr(self.real, name)

        def call(*args):
            self.calls.append((name, args))
            if self.launch is not None:
                self.launch(name, args)
            return 0
        return call


@pytest.fixture
def library(monkeypatch):
    lib = StandIn(sw.lib())
    for m in (sw, sw.train, sw.lora):
        monkeypatch.setattr(m, "lib", lambda: lib)
        monkeypatch.setattr(m, "_dev_bf16", lambda t, name: t.data_ptr(), raising=False)
        monkeypatch.setattr(m, "_stream", lambda stream: 0 if stream is None else int(stream))
    monkeypatch.setattr(sw.lora, "_dev_vec", lambda t, dtype, n, name: t.data_ptr())
    return lib


@pytest.mark.parametrize("lead", [(0,), (2, 0), (0, 3)])
@pytest.mark.parametrize("fn", ["kept", "recomputed", "block"])
def test_backward_of_an_empty_batch(library, fn, lead):
    """No rows: an empty gradient of A in A's own shape, gradients for the weights."""
    K, N = 64, 72
    A = torch.zeros(*lead, K, **BF).requires_grad_()
    W = [torch.zeros(*s, **BF).requires_grad_() for s in ((K, N), (K, N), (N, K))]
    if fn == "block":
        out = sw.swiglu_mlp(A, *W)
    else:
        W.pop()
        out = sw.swiglu(A, *W, recompute=fn == "recomputed")
    assert out.shape == (*lead, W[-1].shape[1])
    grads = torch.autograd.grad(out, [A] + W, torch.zeros_like(out))
    assert [g.shape for g in grads] == [t.shape for t in [A] + W]


class Streams:
    """torch's streams by their handles: the current one, the ones under capture, and on
    which each buffer was allocated."""

    def __init__(self, monkeypatch):
        self.current, self.capturing, self.allocated = 3, set(), []
        empty = torch.empty

        class Stream:
            def __init__(self, handle):
                self.cuda_stream = handle

        class Using:
            def __init__(use, stream):
                use.handle = stream.cuda_stream

            def __enter__(use):
                use.before, self.current = self.current, use.handle

            def __exit__(use, *exc):
                self.current = use.before

        def recorded(*args, **kw):
            self.allocated.append(self.current)
            return empty(*args, **kw)

        monkeypatch.setattr(torch, "empty", recorded)
        for name, value in (
                ("current_stream", lambda device=None: Stream(self.current)),
                ("default_stream", lambda device=None: Stream(0)),
                # a handle of 0 gives a stream of the pool, as in torch
                ("ExternalStream", lambda handle, device=None: Stream(handle or 999)),
                ("stream", Using), ("current_device", lambda: 0), ("is_initialized", lambda: True),
                ("is_current_stream_capturing", lambda: self.current in self.capturing)):
            monkeypatch.setattr(torch.cuda, name, value)
        monkeypatch.setattr(sw, "_raw_stream", lambda device: self.current)


@pytest.fixture
def streams(monkeypatch):
    return Streams(monkeypatch)


CPU = torch.device("cpu")


@pytest.mark.parametrize("handle", [0, 3, 7])
def test_buffers_belong_to_the_stream_that_uses_them(streams, handle):
    """Also where that is the default stream, whose handle is 0, and another is current."""
    sw._new((2, 8), CPU, handle, handle)
    sw.Workspace(CPU).get(64, handle)
    assert streams.allocated == [handle, handle] and streams.current == 3


@pytest.mark.parametrize("capturing", [{3, 7}, {7}])
def test_workspace_of_a_captured_stream(streams, capturing):
    """A call on stream 7 under capture, with stream 3 current (the capture forked, or not
    joined by 3): its own buffer of stream 7, never one kept for other calls."""
    streams.capturing = capturing
    first, nbytes = sw._scratch(None, 64, CPU, 7)
    assert nbytes >= 64 and streams.allocated == [7]
    second, _ = sw._scratch(None, 64, CPU, 7)
    assert second.data_ptr() != first.data_ptr() and streams.allocated == [7, 7] and streams.current == 3


# a call's name, and the argument that holds its workspace
WORKSPACE_AT = {"swiglu_train_forward": 9, "swiglu_train_backward": 12, "swiglu_mlp_train_backward": 15,
                "swiglu_fused_packed_lora": 11, "swiglu_gemm_packed_lora": 11, "swiglu_fused_packed": 6,
                "swiglu_gemm_packed": 6, "swiglu_mlp_packed": 8, "swiglu_mlp_down": 6, "swiglu_mlp_unfused": 11}
M, K, N, L, R = 130, 4096, 264, 3, 16   # every product splits K (of 65 rows where it is on its own)


def calls():
    a, y, w, v = (torch.zeros(*s, **BF) for s in ((M, K), (M, N), (K, N), (N, K)))
    wp = torch.zeros(sw.swiglu_packed_bytes(K, N) // 2, **BF)
    wg, vg = (torch.zeros(sw.swiglu_gemm_packed_bytes(*s) // 2, **BF) for s in ((K, N), (N, K)))
    lp = torch.zeros(sw.swiglu_lora_packed_bytes(K, N, L, R) // 2, **BF)
    ids, scales = torch.zeros(M, dtype=torch.int32), torch.ones(L)
    return {"swiglu_train_forward": lambda: sw.swiglu_train_forward(a, w, w),
            "swiglu_train_backward": lambda: sw.swiglu_train_backward(y, a, w, w),
            "swiglu_mlp_train_backward": lambda: sw.swiglu_mlp_train_backward(a, a, w, w, v, y, y, y),
            "swiglu_fused_packed_lora": lambda: sw.swiglu_fused_packed_lora(a, wp, lp, ids, scales, N, R),
            "swiglu_gemm_packed_lora": lambda: sw.swiglu_gemm_packed_lora(a, wg, lp, ids, scales, N, R),
            "swiglu_fused_packed": lambda: sw.swiglu_fused_packed(a, wp, N, variant=sw.VARIANT_SPLIT_K),
            "swiglu_gemm_packed": lambda: sw.swiglu_gemm_packed(a[:65], wg, N),
            "swiglu_mlp_packed": lambda: sw.swiglu_mlp_packed(a, wp, vg, N, variant=sw.VARIANT_SPLIT_K),
            "swiglu_mlp_down": lambda: sw.swiglu_mlp_down(a[:65], wg, N),
            "swiglu_mlp_unfused": lambda: sw.swiglu_mlp_unfused(y[:65], vg, vg, wg, K)}


@pytest.mark.parametrize("name", sorted(WORKSPACE_AT))
def test_threads_do_not_share_a_workspace(library, streams, name):
    """Two threads in the same call on one stream: a call is several launches, and
    another thread's may fall between them, so each call has a buffer of its own."""
    streams.current = 0
    gate = threading.Barrier(2, timeout=60)
    library.launch = lambda fn, args: gate.wait()   # both are in the library at once
    failed = []

    def thread():
        try:
            calls()[name]()
        except Exception as e:   # noqa: BLE001
            failed.append(e)
            gate.abort()

    threads = [threading.Thread(target=thread) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    at = WORKSPACE_AT[name]
    (p, n), (q, m) = [args[at:at + 2] for fn, args in library.calls]
    assert n > 0 and m > 0 and (p + n <= q or q + m <= p), "both at %#x" % p


def test_block_refuses_what_its_backward_pass_would(library):
    """W3 of other columns than A's has no backward pass: refused before the forward pass
    runs where a gradient is wanted, and computed where none is."""
    a, w = torch.zeros(4, 64, **BF), torch.zeros(64, 72, **BF)
    wide = torch.zeros(72, 80, **BF)
    for leaf in (a, w, wide):
        with pytest.raises(ValueError, match=r"W3 must be \[72, 64\] \(got \[72, 80\]\)"):
            sw.swiglu_mlp(*(t.clone().requires_grad_() if t is leaf else t for t in (a, w, w.clone(), wide)))
    assert library.calls == []
    assert sw.swiglu_mlp(a, w, w, wide).shape == (4, 80)
    with torch.no_grad():
        assert sw.swiglu_mlp(a.clone().requires_grad_(), w, w, wide).shape == (4, 80)
