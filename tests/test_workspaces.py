"""Workspaces that calls without one of their own take: on which stream they are allocated, when
they are replaced, and what a capture holds.  The host part runs without a GPU, on stand-ins
for streams and memory."""
import contextlib

import numpy as np
import pytest
import torch

from stochastic_sparse_kv_gb300 import santa, _build, workloads
from tests import kv4_util

DEV = "cuda"
CPU = torch.device("cpu")


class FakeStream:
    def __init__(self, handle, capturing=False):
        self.cuda_stream, self.capturing, self.device = handle, capturing, CPU


class Host:
    """The current stream, what was allocated on which, and what was launched."""

    def __init__(self):
        self.main = self.now = FakeStream(1)
        self.made, self.calls = [], []

    @contextlib.contextmanager
    def stream(self, s):
        before, self.now = self.now, s
        yield
        self.now = before

    def new_workspace(self, nbytes, device, stream=None):
        ws = torch.empty(nbytes, dtype=torch.uint8)
        self.made.append((ws, self.now, stream))
        return ws

    def call(self, stream, n_max):
        """decode_kv4 from the point where its tensors have been checked."""
        q = torch.zeros(1, 8, 128, dtype=torch.bfloat16)
        fn = lambda shape, *a: self.calls.append((a[-1], a[-3])) or 0  # noqa: E731
        santa._window_call(q, (1, 1, n_max, 128, CPU), (None,), fn, "call", torch.zeros(1, dtype=torch.int32), 0, 0, 0.0,
                           torch.empty(1, 8, 128), torch.float32, None, stream)
        return self.calls[-1]


@pytest.fixture
def host(monkeypatch):
    _build.build()
    h = Host()
    monkeypatch.setattr(santa, "_ws_cache", {})
    monkeypatch.setattr(santa, "new_workspace", h.new_workspace)
    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "stream", h.stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: h.now)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: h.now.capturing)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: h.now.cuda_stream, raising=False)
    return h


def test_a_workspace_is_allocated_on_the_stream_that_uses_it(host):
    s = FakeStream(2)
    for n_max in (64, 64, 65536):                 # made, used again, replaced by a larger one
        assert host.call(s, n_max) == (2, host.made[-1][0].data_ptr())
    assert len(host.made) == 2
    assert all(on is s for _, on, _ in host.made)
    assert host.now is host.main
    assert host.call(None, 64)[0] == 1 and host.made[-1][1] is host.main


def test_a_capture_is_asked_of_the_stream_that_is_used(host):
    s = FakeStream(3, capturing=True)
    a, b = host.call(s, 64), host.call(s, 64)
    assert len(host.made) == 2 and a[1] != b[1]   # each of the graph's own
    assert all(on is s for _, on, _ in host.made)
    assert not santa._ws_cache


def test_windowed_calls_leave_the_sampled_ones_workspace(host):
    s = FakeStream(4)
    ws = santa._cached_workspace(100000, CPU, s)
    host.call(s, 65536)
    assert santa._cached_workspace(100000, CPU, s) is ws


def test_a_workspace_that_a_captured_decode_holds_is_never_freed(host, monkeypatch):
    kept = {}
    monkeypatch.setattr(santa, "_ws_captured", kept, raising=False)
    s = FakeStream(5)
    ws = santa._cached_workspace(1000, CPU, s)
    s.capturing = True
    assert santa._cached_workspace(1000, CPU, s) is ws           # no clearing in the graph
    s.capturing = False
    assert santa._cached_workspace(5000, CPU, s) is not ws
    assert any(x is ws for x in kept.values())
    # without one from before, a capture's is its own: the clearing runs with the graph only
    t = FakeStream(6, capturing=True)
    inside = santa._cached_workspace(1000, CPU, t)
    t.capturing = False
    assert santa._cached_workspace(1000, CPU, t) is not inside


@pytest.mark.parametrize("window,sinks", [(1 << 31, 0), ((1 << 32) + 5, 0), (5 - (1 << 32), 0), (4, 5 - (1 << 32))])
def test_windows_that_32_bits_do_not_hold_are_refused(host, window, sinks):
    with pytest.raises(ValueError, match="32-bit"):
        santa._window_call(torch.zeros(1, 8, 128), (1, 1, 64, 128, CPU), (None,), lambda *a: 0, "call",
                           torch.zeros(1, dtype=torch.int32), window, sinks, 0.0, torch.empty(1, 8, 128), torch.float32, None, None)


def test_a_stream_of_another_device_is_refused(monkeypatch):
    class Other:
        cuda_stream, device = 7, torch.device("cuda", 1)

    monkeypatch.setattr(torch.cuda, "Stream", Other)
    with pytest.raises(ValueError, match="stream"):
        santa._current(Other(), torch.device("cuda", 0))


# ------------------------------------------------------------------ on the GPU

def _problem(n, seed, B=2):
    seq = [n - 3 * b for b in range(B)]
    g = torch.Generator().manual_seed(seed)
    q = workloads.make_q(B, 8, 128, 3.0, g).to(DEV)
    k, v = (torch.randn(B, 2, n, 128, generator=g).to(torch.bfloat16) for _ in range(2))
    cache = santa.KV4Cache(*(torch.from_numpy(x).to(DEV) for t in (k, v) for x in kv4_util.quantise(t)))
    return q, k.to(DEV), v.to(DEV), cache, torch.tensor(seq, dtype=torch.int32, device=DEV)


def _ops(p):
    q, k, v, cache, sl = p
    return [lambda **kw: santa.decode_window(q, k, v, sl, 700, 3, **kw), lambda **kw: santa.decode_kv4(q, cache, sl, **kw),
            lambda **kw: santa.decode(q, k, v, sl, 64, "systematic", seed=3, two_pass=True, **kw)[0]]


@pytest.mark.gpu
def test_growing_on_an_explicit_stream_without_synchronising():
    """Ever larger problems on a side stream, beside work on the current one that takes whatever
    memory is free."""
    problems = [_problem(n, n) for n in (64, 608, 2000, 8000)]
    want = [[op().clone() for op in _ops(p)] for p in problems]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        santa._ws_cache.clear()
        got = []
        for p in problems:
            for op in _ops(p):
                got.append(op(stream=side))
                for mb in (1, 4, 16, 32):
                    torch.full((mb << 18,), 7.0, device=DEV)
        torch.cuda.synchronize()
        for a, b in zip(got, [x for w in want for x in w]):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_streams_given_as_handles_and_plans_on_a_stream():
    """Any object that holds a CUDA stream handle will do, and a plan keeps to its stream."""
    class Handle:
        def __init__(self, s):
            self.cuda_stream = s.cuda_stream

    p = _problem(2000, 8)
    want = [op().clone() for op in _ops(p)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for s in (Handle(side), torch.cuda.ExternalStream(side.cuda_stream), side):
        got = [op(stream=s) for op in _ops(p)]
        assert santa.new_workspace(70000, DEV, s).numel() == 70000
        side.synchronize()
        assert all(torch.equal(a, w) for a, w in zip(got, want))
    q, k, v, _, sl = p
    plan = santa.DecodePlan(q, k, v, sl, 64, "systematic", two_pass=True, stream=side)
    _ops(_problem(8000, 9))[2](stream=side)              # a larger call on the plan's stream
    out, _ = plan(3)
    side.synchronize()
    assert torch.equal(out, want[2])


@pytest.mark.gpu
def test_draws_on_an_explicit_stream_use_memory_of_that_stream():
    """Memory that work still running on the current stream has given back is not written by another stream."""
    q = workloads.make_q(64, 32, 128, 3.0, torch.Generator().manual_seed(1)).to(DEV)
    calls = [lambda **kw: santa.sample_points(64, 32, 256, "stratified", 7, **kw), lambda **kw: santa.ternary_query(q, 7, **kw)]
    want = [c().clone() for c in calls]
    side = torch.cuda.Stream()
    big = torch.ones(1 << 28, device=DEV)
    torch.cuda.synchronize()
    for c, w in zip(calls, want):
        for _ in range(4):
            for _ in range(20):
                big.mul_(1.0)                                    # the current stream is busy
            gone = torch.full_like(w, 3)                         # written late, given back at once
            at = gone.data_ptr()
            del gone
            got = c(stream=side)
            assert got.data_ptr() != at
            torch.cuda.synchronize()
            assert torch.equal(got, w)


@pytest.mark.gpu
def test_two_captured_branches_with_explicit_streams():
    """Two branches of one graph, forked from the captured stream, each a call on its own stream."""
    p, r = _problem(4000, 1), _problem(3008, 2)
    ops = [_ops(p)[0], _ops(p)[1], _ops(r)[1], _ops(r)[0]]
    outs = [torch.zeros(2, 8, 128, device=DEV) for _ in ops]
    want = [op().clone() for op in ops]
    main, s1, s2 = (torch.cuda.Stream() for _ in range(3))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        for s in (s1, s2):
            s.wait_stream(main)
        for i, op in enumerate(ops):
            op(stream=(s1, s2)[i % 2], out=outs[i])
        for s in (s1, s2):
            main.wait_stream(s)
    for _ in range(5):
        for o in outs:
            o.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)


@pytest.mark.gpu
def test_a_captured_decode_outlives_larger_calls_on_its_stream():
    p, big = _problem(1000, 4), _problem(8000, 5)
    out = torch.zeros(2, 8, 128, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    sampled = _ops(p)[2]
    with torch.cuda.stream(s):
        want = sampled().clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        sampled(out=out)
    with torch.cuda.stream(s):
        wants = [op().clone() for op in _ops(big)]
        fill = [torch.full((4 << 18,), 7.0, device=DEV) for _ in range(16)]
        for _ in range(3):
            graph.replay()
            assert all(torch.equal(op(), w) for op, w in zip(_ops(big), wants))
    torch.cuda.synchronize()
    assert torch.equal(out, want) and all(bool((f == 7).all()) for f in fill)


@pytest.mark.gpu
def test_a_first_call_inside_a_capture_leaves_the_stream_usable():
    """Captured without a call before: the clearing of the graph's workspace runs with the graph,
    and calls on the stream outside it do not use that workspace."""
    p = _problem(784, 6)
    want = [op().clone() for op in _ops(p)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [torch.zeros(2, 8, 128, device=DEV) for _ in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        for op, o in zip(_ops(p), outs):
            op(out=o)
    with torch.cuda.stream(s):
        got = [op() for op in _ops(p)]
        graph.replay()
    torch.cuda.synchronize()
    for a, b, w in zip(got, outs, want):
        assert torch.equal(a, w) and torch.equal(b, w)
    assert np.isfinite(want[0].cpu().numpy()).all()
