"""Whose memory a call on a given stream uses: what the binding allocates for it, results and scratch,
has to come from that stream's pool, since the allocator orders the reuse of a block on the stream
it was made on."""
import contextlib
import math
from types import SimpleNamespace

import pytest
import torch

import fused_reference as R

SIDE = 0x7000       # a stream's handle on the CPU: nothing is launched


# ---------------------------------------------------------------------------
# CPU: the stream that is current at each allocation, with stand-ins for tensors and library
# ---------------------------------------------------------------------------

class Log:
    def __init__(self):
        self.current = 0
        self.made = []          # (shape, current stream) of every allocation


class Fake:
    """The part of a CUDA tensor that the binding looks at."""
    is_cuda = True
    device = torch.device("cuda", 0)

    def __init__(self, log, shape, dtype):
        self.log, self.shape, self.dtype = log, torch.Size(shape), dtype

    def get_device(self):
        return 0

    def dim(self):
        return len(self.shape)

    def stride(self):
        return tuple(math.prod(self.shape[i + 1:]) for i in range(len(self.shape)))

    def is_contiguous(self):
        return True

    def numel(self):
        return math.prod(self.shape)

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        return 0x10000

    def record_stream(self, stream):
        pass

    def new_empty(self, shape, dtype=None):
        shape = (shape,) if isinstance(shape, int) else shape
        self.log.made.append((tuple(shape), self.log.current))
        return Fake(self.log, shape, dtype or self.dtype)

    def new_empty_strided(self, shape, stride, dtype=None):
        return self.new_empty(shape, dtype)

    def unbind(self):
        return [Fake(self.log, self.shape[1:], self.dtype) for _ in range(self.shape[0])]

    def view(self, dtype):
        return Fake(self.log, self.shape, dtype)

    def flatten(self):
        return Fake(self.log, (self.numel(),), self.dtype)


@pytest.fixture
def fakes(monkeypatch):
    from bit_weight_only_linear_b200 import awq
    log = Log()

    @contextlib.contextmanager
    def stream(s):
        before, log.current = log.current, s.cuda_stream
        yield
        log.current = before

    calls = []

    class Library:
        def __getattr__(self, name):
            if name.endswith("workspace_bytes"):
                return lambda *a: 4096
            return lambda *a: calls.append((name, a[-1])) or 0

    monkeypatch.setattr(awq, "_lib", Library())
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: SimpleNamespace(cuda_stream=h))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: SimpleNamespace(cuda_stream=log.current))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: log.current, raising=False)
    monkeypatch.setattr(torch, "empty", lambda *shape, dtype=None, device=None: Fake(log, (0,), torch.uint8).new_empty(
        shape[0] if isinstance(shape[0], (tuple, list)) else shape, dtype))
    monkeypatch.setattr(torch, "empty_like", lambda x: x.new_empty(x.shape))

    def tensor(*shape, dtype=torch.float16):
        return Fake(log, shape, dtype)
    return awq, log, tensor, calls


def _new_calls(awq, t, stream):
    w = (t(64, 32, dtype=torch.int32), t(64, 2), t(64, 1, dtype=torch.int32))
    e = tuple(t(2, *x.shape, dtype=x.dtype) for x in w)
    offsets, rows = t(3, dtype=torch.int32), t(300, dtype=torch.int32)
    return {
        "linear_fused": lambda: awq.linear_fused(t(4, 256), *w, 128, True, stream=stream),
        "linear_grouped": lambda: awq.linear_grouped(t(9, 256), *e, offsets, rows, 128, True, stream=stream),
        "moe_route": lambda: awq.moe_route(t(100, 8, dtype=torch.float32), 2, stream=stream),
        "moe_combine": lambda: awq.moe_combine(t(8, 64), t(4, 2, dtype=torch.float32), t(4, 2, dtype=torch.int32),
                                               stream=stream),
    }


NEW = {"linear_fused": 1, "linear_grouped": 2, "moe_route": 3, "moe_combine": 1}     # allocations of a call


@pytest.mark.parametrize("name", NEW)
@pytest.mark.parametrize("stream", [SIDE, 0, None])
def test_allocations_of_the_fused_operators_belong_to_the_stream(fakes, name, stream):
    awq, log, t, calls = fakes
    log.current = 0 if stream is None else 0x9000        # another stream is current
    _new_calls(awq, t, stream)[name]()
    want = 0 if stream is None else stream
    assert [s for _, s in log.made] == [want] * NEW[name]
    assert calls == [("awq_" + name, want)]


def _older_calls(awq, t, stream):
    X, W = t(64, 256), t(64, 256)
    w = (t(64, 32, dtype=torch.int32), t(64, 2), t(64, 1, dtype=torch.int32))
    return {
        "quantize_pack": lambda: awq.quantize_pack(W, None, 128, True, stream=stream),
        "fold_inverse_scale": lambda: awq.fold_inverse_scale(X, t(256), stream=stream),
        "linear_gemv": lambda: awq.linear_gemv(t(4, 256), *w, 128, True, stream=stream),
        "linear_gemm": lambda: awq.linear_gemm(X, *w, 128, True, stream=stream),
        "scale_search": lambda: awq.scale_search(X, W, 128, True, stream=stream),
        "scale_search_noalloc": lambda: awq.scale_search_noalloc(X, W, 128, True, stream=stream),
        "apply_clip": lambda: awq.apply_clip(X, W, None, 128, True, stream=stream, errors=True),
    }


OLDER = {"quantize_pack": 3, "fold_inverse_scale": 1, "linear_gemv": 1, "linear_gemm": 2, "scale_search": 4,
         "scale_search_noalloc": 3, "apply_clip": 6}


@pytest.mark.parametrize("name", OLDER)
@pytest.mark.parametrize("stream", [SIDE, 0, None])
def test_allocations_of_the_other_calls_belong_to_the_stream(fakes, monkeypatch, name, stream):
    awq, log, t, calls = fakes
    monkeypatch.setattr(awq, "_GEMM_WS", {})
    log.current = 0 if stream is None else 0x9000
    _older_calls(awq, t, stream)[name]()
    want = 0 if stream is None else stream
    assert [s for _, s in log.made] == [want] * OLDER[name]
    assert calls == [("awq_" + name, want)]


def test_gemm_workspaces_of_two_streams_differ(fakes, monkeypatch):
    awq, log, t, _ = fakes
    monkeypatch.setattr(awq, "_GEMM_WS", {})
    a, b, again = (awq.gemm_workspace(64, 64, 256, stream=s, device=0) for s in (SIDE, 0, SIDE))
    assert a is not b and again is a
    # a captured call's belongs to its graph: neither kept nor taken from the eager calls
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    c, d = (awq.gemm_workspace(64, 64, 256, stream=SIDE, device=0) for _ in range(2))
    assert c is not a and c is not d and len(awq._GEMM_WS) == 2


# ---------------------------------------------------------------------------
# GPU
# ---------------------------------------------------------------------------

def _pool(t):
    """The stream whose pool holds a tensor's memory."""
    p = t.data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= p < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not in the allocator's segments")


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True])
def test_results_belong_to_the_given_stream(lib, handle):
    s = torch.cuda.Stream()
    st = s.cuda_stream if handle else s
    w, we = R.packed(1, 64, 256, 64, True), R.packed(2, 64, 256, 64, True, lead=(2,))
    X = R.activations(3, 300, 256)
    logits = torch.randn(300, 2, generator=torch.Generator().manual_seed(4)).cuda()
    torch.cuda.synchronize()
    r = lib.moe_route(logits, 1, stream=st)
    h = lib.linear_grouped(X, *we, r.offsets, r.rows, 64, True, stream=st)
    made = [lib.linear_fused(X, *w, 64, True, stream=st), h, lib.moe_combine(h, r.weights, r.positions, stream=st), *r]
    s.synchronize()
    lib.device_error()
    assert all(_pool(t) == s.cuda_stream for t in made)
    assert _pool(lib.linear_fused(X, *w, 64, True)) == torch.cuda.current_stream().cuda_stream


@pytest.mark.gpu
def test_calls_on_a_side_stream_leave_the_current_streams_blocks(lib):
    """Blocks freed on the current stream, with work that reads and writes them still queued there: a routed
    and gathered product on a side stream, whose scratch and results have the sizes of those blocks."""
    T, E, k, N, K, G = 512, 4, 2, 128, 512, 64
    w = R.packed(5, N, K, G, True, lead=(E,))
    X = R.activations(6, T, K)
    logits = torch.randn(T, E, generator=torch.Generator().manual_seed(7)).cuda()
    r0 = lib.moe_route(logits, k)
    y0 = lib.linear_grouped(X, *w, r0.offsets, r0.rows, G, True)
    c0 = lib.moe_combine(y0, r0.weights, r0.positions)
    need = lib.load_library().awq_linear_grouped_workspace_bytes(T * k, E, K)
    sizes = [need, T * k * N * 2, T * N * 2, 4 * T * k * 4, 4 * (E + 1),
             lib.load_library().awq_moe_route_workspace_bytes(T, E)]
    kept = [torch.zeros(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    blocks = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)                      # about 0.1 s
    for a, b in zip(kept, blocks):
        a.copy_(b)
        b.fill_(255)
    del a, b, blocks                                    # free for the current stream, not for another
    r = lib.moe_route(logits, k, stream=s)
    y = lib.linear_grouped(X, *w, r.offsets, r.rows, G, True, stream=s)
    c = lib.moe_combine(y, r.weights, r.positions, stream=s)
    torch.cuda.synchronize()
    lib.device_error()
    assert all((a == 7).all() for a in kept)
    assert all(torch.equal(a, b) for a, b in zip(r, r0)) and torch.equal(y, y0) and torch.equal(c, c0)


@pytest.mark.gpu
def test_two_batches_on_two_streams_with_split_sums(lib):
    """linear_gemm splits K over a workspace: overlapping calls of two streams do not share it."""
    N, K, G = 512, 4096, 128
    w = R.packed(8, N, K, G, True)
    X = [R.activations(9 + i, 64, K) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in X]
    want = [lib.linear_gemm(x, *w, G, True) for x in X]
    assert lib.gemm_workspace(64, N, K, G, True) is not None
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            outs[i].append(lib.linear_gemm(X[i], *w, G, True, stream=s))
    torch.cuda.synchronize()
    lib.device_error()
    assert all(torch.equal(y, want[i]) for i in range(2) for y in outs[i])


@pytest.mark.gpu
def test_two_captured_batches_replayed_at_once(lib):
    """Graphs of split products, one of each stream and an eager call beside them."""
    N, K, G = 512, 4096, 128
    w = R.packed(8, N, K, G, True)
    X = [R.activations(11 + i, 64, K) for i in range(3)]
    want = [lib.linear_gemm(x, *w, G, True) for x in X]
    side = torch.cuda.Stream()
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(lib.linear_gemm(X[i], *w, G, True))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        eager = lib.linear_gemm(X[2], *w, G, True)
    torch.cuda.synchronize()
    lib.device_error()
    assert torch.equal(eager, want[2]) and all(torch.equal(o, y) for o, y in zip(outs, want))
