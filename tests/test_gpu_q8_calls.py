"""Calls of the 8-bit history's attention side by side (GPU; calls the C ABI through the binding):
streams, host threads and captured graphs at once, each with inputs and sizes of its own, the
scratch left to the binding.  Every result has to be, bit for bit, what the same call gives alone
with a workspace of its own.
"""
import threading

import pytest
import torch

from long_context_speculative_gb300 import rapid

import _q8

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def _no_error_bits():
    torch.cuda.synchronize()
    rapid.rapid_device_error(True)
    yield
    torch.cuda.synchronize()
    assert rapid.rapid_device_error(True) == 0


class Call:
    """One call's inputs and what it gives alone."""

    def __init__(self, seed, B=1, Hq=8, Hkv=2, n=11, blocks=400, tail=37):
        c = _q8.cache(B, Hkv, 128, BF16, [blocks - 7 * b for b in range(B)], [tail] * B, n, seed=seed)
        self.c = {k: v.to(DEV) for k, v in c.items()}
        g = torch.Generator().manual_seed(seed)
        self.Q = torch.randn((B, Hq, n, 128), generator=g).to(BF16).to(DEV)
        nbytes = rapid.rapid_verify_attn_q8_workspace_size(
            B, Hq, Hkv, 128, n, self.c["K"].shape[2], self.c["page_table"].shape[1], rapid._dtype_code(self.Q))
        self.alone = self.run(workspace=torch.empty(nbytes, dtype=torch.uint8, device=DEV))
        torch.cuda.synchronize()

    def run(self, **kw):
        c = self.c
        return rapid.verify_attn_q8(self.Q, c["K"], c["V"], c["pages"], c["scales"], c["page_table"],
                                    c["sealed_len"], c["tail_len"], **kw)

    def check(self, got, what):
        for x, y in zip(got, self.alone):
            assert torch.equal(x, y), what


def _mix():
    # different sizes of scratch and of work
    return [Call(1), Call(2, B=4, n=6, blocks=90), Call(3, Hq=28, Hkv=2, n=32, blocks=200), Call(4, Hkv=1, n=1, blocks=30)]


def test_two_streams_take_turns_without_waiting():
    calls, streams = _mix(), [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(40):
        for s, stream in enumerate(streams):
            c = calls[(i + 2 * s + i // 7) % 4]
            got.append((c, c.run(stream=stream)))
    torch.cuda.synchronize()
    for i, (c, r) in enumerate(got):
        c.check(r, i)


def test_scratch_that_grows_while_work_is_pending():
    small, large = Call(5, Hkv=1, n=1, blocks=40), Call(6, Hq=28, Hkv=4, n=32, B=2, blocks=150)
    stream = torch.cuda.Stream()                       # a stream whose scratch starts empty
    got = [(c, c.run(stream=stream)) for c in (small, small, large, small, large, large, small)]
    torch.cuda.synchronize()
    for i, (c, r) in enumerate(got):
        c.check(r, i)


def test_two_host_threads_on_one_stream():
    calls, stream = _mix(), torch.cuda.Stream()
    got, lock, go = [], threading.Lock(), threading.Barrier(2)

    def work(k):
        go.wait()
        for i in range(30):
            c = calls[(2 * k + i) % 4]
            r = c.run(stream=stream)
            with lock:
                got.append((c, r))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert len(got) == 60
    for i, (c, r) in enumerate(got):
        c.check(r, i)


def test_graphs_and_eager_calls_at_once():
    a, b, eager = Call(7), Call(8, B=4, n=6, blocks=90), Call(9, Hq=28, Hkv=2, n=32, blocks=200)
    graphs = []
    for c in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r = c.run()
        graphs.append((c, g, r))
    streams = [torch.cuda.Stream() for _ in range(2)]
    main = torch.cuda.current_stream()
    got = []
    for _ in range(12):
        for (c, g, r), stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                g.replay()
        got.append(eager.run())
        got.append(eager.run(stream=streams[0]))
    torch.cuda.synchronize()
    assert main == torch.cuda.current_stream()
    for c, _, r in graphs:
        c.check(r, "graph")
    for i, r in enumerate(got):
        eager.check(r, i)
