"""Calls captured into CUDA graphs (GPU): what they report, which memory they
use, and for how long it is theirs."""

import gc
import threading
import time

import pytest
import torch

import paged_kv_cache_471_b200 as pa
from kv_reference import Cache, attention

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def queries(T, Hq, D, seed=2):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((T, Hq, D), generator=g).to(torch.bfloat16)


class Setup:
    """A long sequence whose decode and prefill split the keys."""
    Hk, Hq, D, B = 2, 8, 128, 16

    def __init__(self, kv="int8_block", lens=(6000,), seed=13):
        self.kv = kv
        self.cache = Cache(kv, list(lens), self.Hk, self.D, self.B, seed=seed)
        self.kc, self.vc = self.cache.packed(DEV)
        self.ks, self.vs = self.cache.scales(DEV)
        self.bt, self.sl = self.cache.tables.to(DEV), self.cache.lens.to(DEV)
        self.max_len = max(lens)

    def decode(self, out, q, **kw):
        pa.decode(out, q, self.kc, self.vc, self.Hk, 0.09, self.bt, self.sl, self.B, self.max_len,
                  self.kv, self.ks, self.vs, **kw)

    def prefill(self, out, q, start, **kw):
        pa.prefill(out, q, self.kc, self.vc, self.Hk, 0.09, self.bt, self.sl, start, self.B,
                   self.max_len, self.kv, self.ks, self.vs, **kw)

    def check(self, out, q, start):
        ref, tol = attention(self.cache, q.cpu(), start, 0.09)
        err = (out.cpu().double() - ref).abs()
        assert (err <= tol).all(), float((err / tol.clamp(min=1e-300)).max())


def capture(fn, **kw):
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st, **kw):
        fn()
    torch.cuda.synchronize()
    return graph


def let_go(keys):
    """Whether the workspaces of these captures are let go in a while (a graph's
    objects are destroyed on a thread of the driver)."""
    for _ in range(100):
        gc.collect()
        pa.read_status(device=DEV)
        if not keys & set(pa._captured):
            return True
        time.sleep(0.05)
    return False


@pytest.mark.parametrize("op", ["decode", "decode balanced", "prefill"])
def test_a_replay_s_errors_are_read(op):
    """Bad device data met by a replay sets its bits where read_status finds
    them, at each replay until they are cleared, also once the graph is gone."""
    s = Setup(lens=(6000, 40))
    if op == "prefill":
        q = queries(9, s.Hq, s.D).to(DEV)
        out, start = torch.empty_like(q), torch.tensor([0, 5, 9], dtype=torch.int32, device=DEV)
        fn = lambda: s.prefill(out, q, start)
    else:
        q = queries(2, s.Hq, s.D).to(DEV)
        out = torch.empty_like(q)
        kw = {} if op == "decode" else dict(schedule="balanced")
        fn = lambda: s.decode(out, q, **kw)
    before = set(pa._captured)
    graph = capture(fn)
    mine = set(pa._captured) - before
    assert len(mine) == 1
    pa.read_status(device=DEV, clear=True)
    graph.replay()
    assert pa.read_status(device=DEV) == 0
    last = (6000 - 1) // s.B
    good = int(s.bt[0, last])
    s.bt[0, last] = s.cache.num_blocks + 5
    graph.replay()
    assert pa.read_status(device=DEV) == pa.PA_DEV_BAD_BLOCK_ID
    s.bt[0, last] = good
    graph.replay()  # the bits stay
    assert pa.read_status(device=DEV, clear=True) == pa.PA_DEV_BAD_BLOCK_ID
    graph.replay()
    assert pa.read_status(device=DEV) == 0
    s.bt[0, last] = -1
    graph.replay()
    assert mine <= set(pa._captured)
    del graph
    assert let_go(mine)
    assert pa.read_status(device=DEV, clear=True) == pa.PA_DEV_BAD_BLOCK_ID
    assert pa.read_status(device=DEV) == 0


def test_a_replay_clears_nothing():
    """The workspace of a graph is zeroed once: what lies behind the partials of
    its calls, and its status word, are as before after a replay."""
    s = Setup()
    q = queries(1, s.Hq, s.D)
    q_dev = q.to(DEV)
    out = torch.empty_like(q_dev)
    held = []

    def fn():
        held.append(pa.workspace(4 << 20, DEV))
        s.decode(out, q_dev)
        held.append(pa.workspace(256, DEV))

    graph = capture(fn)
    assert held[0].data_ptr() == held[1].data_ptr() and not held[0].any()
    need = pa.workspace_size(1, s.Hq, s.Hk, s.D, s.B, 6000, s.kv)
    assert need < held[0].numel() // 2
    held[0][need:] = 0xA5
    held[0][0] = pa.PA_DEV_PREFIX_MISMATCH
    for _ in range(2):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        s.check(out, q, torch.arange(2))
        assert (held[0][need:] == 0xA5).all()
    assert pa.read_status(device=DEV, clear=True) & pa.PA_DEV_PREFIX_MISMATCH


def test_graphs_streams_and_eager_calls_have_a_workspace_each():
    """Also graphs captured on one stream, and the branches of one graph."""
    st, side = torch.cuda.Stream(), torch.cuda.Stream()
    seen = []
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            seen.append(pa.workspace(5000, DEV))
            side.wait_stream(st)
            with torch.cuda.stream(side):
                seen.append(pa.workspace(5000, DEV))
            seen.append(pa.workspace(5000, DEV, stream=side))
            torch.zeros(1, device=DEV)
            st.wait_stream(side)
        graphs.append(g)
    with torch.cuda.stream(st):
        seen.append(pa.workspace(5000, DEV))
    where = [w.data_ptr() for w in seen]
    assert where[1] == where[2] and where[4] == where[5]
    assert len(set(where)) == 5
    assert all(not w.any() for w in seen)


def test_captures_that_torch_does_not_know_of():
    """A capture begun through the CUDA runtime: torch's allocator does not know
    that the graph keeps addresses, so nothing that it frees may be among them."""
    rt = pytest.importorskip("cuda.bindings.runtime")

    def ok(r):
        assert r[0] == rt.cudaError_t.cudaSuccess, r
        return r[1] if len(r) == 2 else r[1:]

    s = Setup()
    q = queries(1, s.Hq, s.D)
    q_dev = q.to(DEV)
    out = torch.empty_like(q_dev)
    s.decode(torch.empty_like(q_dev), q_dev)  # (as a program warms up)
    torch.cuda.synchronize()
    st, before = torch.cuda.Stream(), set(pa._captured)
    ok(rt.cudaStreamBeginCapture(st.cuda_stream,
                                 rt.cudaStreamCaptureMode.cudaStreamCaptureModeGlobal))
    s.decode(out, q_dev, stream=st)
    graph = ok(rt.cudaStreamEndCapture(st.cuda_stream))
    run = ok(rt.cudaGraphInstantiate(graph, 0))
    ok(rt.cudaGraphDestroy(graph))
    need = pa.workspace_size(1, s.Hq, s.Hk, s.D, s.B, 6000, s.kv)
    others = []
    for stream in (st, torch.cuda.current_stream()):
        with torch.cuda.stream(stream):
            others += [torch.full((need,), 0x3C, dtype=torch.uint8, device=DEV) for _ in range(20)]
    torch.cuda.synchronize()
    ok(rt.cudaGraphLaunch(run, st.cuda_stream))
    torch.cuda.synchronize()
    s.check(out, q, torch.arange(2))
    assert all((t == 0x3C).all() for t in others)
    mine = set(pa._captured) - before
    assert len(mine) == 1
    ok(rt.cudaGraphExecDestroy(run))
    assert let_go(mine)


def test_an_abandoned_capture_keeps_nothing():
    s = Setup()
    q = queries(1, s.Hq, s.D).to(DEV)
    before, mine = set(pa._captured), set()
    with pytest.raises(RuntimeError, match="given up"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            s.decode(torch.empty_like(q), q)
            mine |= set(pa._captured) - before
            raise RuntimeError("given up")
    assert len(mine) == 1 and let_go(mine)


@pytest.mark.parametrize("current", [True, False])
def test_a_first_append_in_a_capture_reports(monkeypatch, current):
    """The first append of a process, captured on the current stream or on one
    that is given: the capture holds, and its replays' errors are read."""
    monkeypatch.setattr(pa, "_status_words", {})
    s = Setup(lens=(40, 17))
    k = queries(2, s.Hk, s.D).to(DEV)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        graph.capture_begin()
        if current:
            pa.append_kv(s.kc, s.vc, k, k, s.bt, s.sl, s.B, s.kv, s.ks, s.vs)
    if not current:
        pa.append_kv(s.kc, s.vc, k, k, s.bt, s.sl, s.B, s.kv, s.ks, s.vs, stream=st)
    with torch.cuda.stream(st):
        graph.capture_end()
    pa.read_status(device=DEV, clear=True)
    graph.replay()
    assert pa.read_status(device=DEV) == 0
    s.bt[0, 2] = s.cache.num_blocks
    graph.replay()
    assert pa.read_status(device=DEV, clear=True) == pa.PA_DEV_BAD_BLOCK_ID


def test_first_appends_of_two_threads_share_a_word(monkeypatch):
    """Both threads' errors are read: each makes another one."""
    for _ in range(20):
        monkeypatch.setattr(pa, "_status_words", {})
        s = Setup(lens=(40, 17), kv="bf16")
        k = queries(2, s.Hk, s.D).to(DEV)
        too_long = s.sl.clone()
        too_long[0] = 1000
        bad = s.bt.clone()
        bad[1, 1] = -1
        torch.cuda.synchronize()
        gate = threading.Barrier(2)
        failed = []

        def call(tables, lens):
            try:
                with torch.cuda.stream(torch.cuda.Stream()):
                    gate.wait()
                    pa.append_kv(s.kc, s.vc, k, k, tables, lens, s.B)
            except Exception as e:
                failed.append(e)

        threads = [threading.Thread(target=call, args=a) for a in ((s.bt, too_long), (bad, s.sl))]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert not failed and len(pa._status_words) == 1
        assert pa.read_status(device=DEV, clear=True) == (pa.PA_DEV_SEQ_LEN_OUT_OF_RANGE |
                                                          pa.PA_DEV_BAD_BLOCK_ID)


def test_graphs_that_are_gone_leave_no_memory_behind():
    """Neither by the next capture, nor by the next read of the status."""
    s = Setup()
    q = queries(1, s.Hq, s.D).to(DEV)
    out = torch.empty_like(q)
    size = 64 << 20
    torch.cuda.synchronize()
    before, base = set(pa._captured), torch.cuda.memory_allocated()

    def fn():
        pa.workspace(size, DEV)
        s.decode(out, q)

    for _ in range(12):
        graph = capture(fn)
        graph.replay()
        mine = set(pa._captured) - before
        del graph
        gc.collect()
        assert let_go(mine)
        assert torch.cuda.memory_allocated() < base + size
