"""The latent cache's operators together, as a decode loop uses them (GPU; calls the C ABI through the
binding).

A prompt enters in chunks: append, read the history's rows back, expand them into keys and values of
every head, expanded attention.  Then verify steps run: append the nodes' rows, absorbed attention
on every layer, acceptance, commit of the accepted path, advance.  Every number a step needs is in
device memory, so the same step captured once in a CUDA graph and replayed has to give the eager
loop's bits.
"""
import threading

import pytest
import torch

from long_context_speculative_gb300 import rapid
from long_context_speculative_gb300 import workloads as wl

import _latent

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16
B, H, NQ, LAYERS, V, CAP = 2, 4, 6, 2, 2000, 512
CHUNKS = (150, 41)


@pytest.fixture(autouse=True)
def _no_error_bits():
    torch.cuda.synchronize()
    rapid.rapid_device_error(True)
    yield
    torch.cuda.synchronize()
    assert rapid.rapid_device_error(True) == 0


class Loop:
    def __init__(self, q8):
        g = torch.Generator().manual_seed(3)
        width, dt = (_latent.Q8_ROW, torch.uint8) if q8 else (_latent.DK, BF16)
        self.cache = [torch.zeros((B, CAP, width), dtype=dt, device=DEV) for _ in range(LAYERS)]
        self.length = torch.zeros(B, dtype=torch.int32, device=DEV)
        self.inv_freq = (5e5 ** (-torch.arange(0, 64, 2).double() / 64)).float().to(DEV)
        self.weight = (1 + 0.1 * torch.randn(512, generator=g)).to(BF16).to(DEV)
        self.up_k, self.up_v = (torch.randn((2, LAYERS, H, 128, 512), generator=g) / 22).to(BF16).to(DEV)
        self.table = rapid.LatentLayerTable(self.cache)

    def append(self, layer, x, q_out, offsets=None):
        """x: latent rows [B, n, 576] and queries [B, n, H, 192] of a layer."""
        kv, q = x
        rapid.latent_append(kv[layer], self.cache[layer], self.length, self.inv_freq,
                            q=q[layer][..., 128:], q_out=q_out, kv_weight=self.weight, row_offset=offsets)

    def absorb(self, layer, q, Q):
        """The queries' plain part through the key expansion, into Q [B, H, n, 576]."""
        Q[..., :512] = torch.einsum("bihd,hdc->bhic", q[layer][..., :128], self.up_k[layer])


def _rows(g, n):
    return (torch.randn((LAYERS, B, n, 576), generator=g).to(BF16).to(DEV),
            torch.randn((LAYERS, B, n, H, 192), generator=g).to(BF16).to(DEV))


def _prompt(loop, g):
    at = 0
    for n in CHUNKS:
        kv, q = x = _rows(g, n)
        for layer in range(LAYERS):
            loop.append(layer, x, q[layer][..., 128:])           # rotated in place
            rows = rapid.latent_read(loop.cache[layer], None, at + n)
            K = torch.einsum("bjc,hdc->bjhd", rows[..., :512], loop.up_k[layer])
            Vv = torch.einsum("bjc,hdc->bjhd", rows[..., :512], loop.up_v[layer])
            O, L = rapid.latent_prefill_attn(q[layer], K, Vv, rows[..., 512:], loop.length)
            want, wl_, eO, eL = _latent.prefill(q[layer], K, Vv, rows[..., 512:], loop.length)
            assert ((O.double() - want).abs() <= eO).all() and ((L.double() - wl_).abs() <= eL).all()
            assert torch.equal(_latent.values(loop.cache[layer][:, :at + n]).to(BF16), rows)
        loop.length += n
        at += n


def _steps(g, n, tree):
    steps = []
    for _ in range(n):
        parents = [wl.random_tree(NQ, 4, g) if tree else wl.chain_parents(NQ) for _ in range(B)]
        depth = torch.zeros((B, NQ), dtype=torch.int32)
        for b in range(B):
            for i in range(1, NQ):
                depth[b, i] = depth[b, parents[b][i]] + 1
        z = torch.randn((B, NQ, V), generator=g) * 2
        q = torch.softmax(z + 0.3 * torch.randn((B, NQ, V), generator=g), -1)
        tok = torch.zeros((B, NQ), dtype=torch.int32)
        for b in range(B):
            for i in range(1, NQ):
                tok[b, i] = int(torch.multinomial(q[b, parents[b][i]], 1, generator=g))
        par = torch.tensor(parents, dtype=torch.int32)
        par[:, 0] = -1
        kv, qq = _rows(g, NQ)
        steps.append(dict(kv=kv, qq=qq, depth=depth.to(DEV),
                          mask=torch.stack([wl.ancestor_mask(p) for p in parents]).to(DEV),
                          z=z.to(DEV), q=q.to(DEV), tok=tok.to(DEV), par=par.to(DEV)))
    return steps


def _step(loop, s, Q, O, L, seed, ws=None):
    for layer in range(LAYERS):
        loop.absorb(layer, s["qq"], Q[layer])
        loop.append(layer, (s["kv"], s["qq"]), Q[layer][..., 512:].transpose(1, 2), s["depth"])
        rapid.latent_attn(Q[layer], loop.cache[layer], loop.length, s["mask"], out=O[layer], lse=L[layer],
                          workspace=ws)
    res = rapid.accept(s["z"], s["q"], s["tok"], s["par"], seed=seed)
    loop.table.commit(loop.length, res["path"], res["n_accepted"])
    rapid.rapid_kv_advance(loop.length, res["n_accepted"], NQ, CAP)
    return res


def _buffers():
    return (torch.zeros((LAYERS, B, H, NQ, 576), dtype=BF16, device=DEV),
            torch.zeros((LAYERS, B, H, NQ, 512), dtype=BF16, device=DEV),
            torch.zeros((LAYERS, B, H, NQ), device=DEV))


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("tree", [False, True])
def test_decode_loop(q8, tree):
    g = torch.Generator().manual_seed(17 + tree)
    loop = Loop(q8)
    _prompt(loop, g)
    Q, O, L = _buffers()
    moved = 0
    for i, s in enumerate(_steps(g, 5, tree)):
        P = loop.length.tolist()
        Ps = [c.clone() for c in loop.cache]
        res = _step(loop, s, Q, O, L, seed=100 + i)
        acc, path = res["n_accepted"].tolist(), res["path"].tolist()
        for layer in range(LAYERS):
            # the cache as attention saw it: the loop's, with the committed rows where they were
            seen = loop.cache[layer].clone()
            for b in range(B):
                # rows before the step never change
                assert torch.equal(seen[b, :P[b]], Ps[layer][b, :P[b]])
            again = Loop(q8)
            again.cache = [c.clone() for c in Ps]
            again.length = torch.tensor(P, dtype=torch.int32, device=DEV)
            again.append(layer, (s["kv"], s["qq"]), torch.empty((B, NQ, H, 64), dtype=BF16, device=DEV), s["depth"])
            before = again.cache[layer]
            want, lw, eO, eL = _latent.attn(Q[layer], before, P, s["mask"])
            assert ((O[layer].double() - want).abs() <= eO).all()
            assert ((L[layer].double() - lw).abs() <= eL).all()
            for b in range(B):
                for k in range(acc[b]):
                    assert torch.equal(seen[b, P[b] + 1 + k], before[b, P[b] + path[b][k]])
                    moved += path[b][k] != k + 1
        assert loop.length.tolist() == [p + 1 + a for p, a in zip(P, acc)]
    assert moved > 0 or not tree


@pytest.mark.parametrize("q8", [False, True])
def test_captured_step_replays_the_eager_loop(q8):
    g = torch.Generator().manual_seed(5)
    eager, graphed = Loop(q8), Loop(q8)
    state = g.get_state()
    _prompt(eager, g)
    g.set_state(state)
    _prompt(graphed, g)
    steps = _steps(g, 4, True)
    Q, O, L = _buffers()
    ref = []
    for i, s in enumerate(steps):
        key = torch.tensor([1000 + i], dtype=torch.int64, device=DEV)
        res = _step(eager, s, Q, O, L, key)
        ref.append((O.clone(), L.clone(), res["next_token"].clone(), eager.length.clone(),
                    [c.clone() for c in eager.cache]))
    # static inputs, one step outside the capture first (on a copy), then replays
    hold = {k: v.clone() for k, v in steps[0].items()}
    key = torch.zeros(1, dtype=torch.int64, device=DEV)
    Q2, O2, L2 = _buffers()
    _step(Loop(q8), hold, Q2, O2, L2, key)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        res = _step(graphed, hold, Q2, O2, L2, key)
    for i, s in enumerate(steps):
        for k, v in s.items():
            hold[k].copy_(v)
        key.fill_(1000 + i)
        graph.replay()
        torch.cuda.synchronize()
        o, l, tok, length, caches = ref[i]
        assert torch.equal(O2, o) and torch.equal(L2, l) and torch.equal(res["next_token"], tok)
        assert torch.equal(graphed.length, length)
        for x, y in zip(graphed.cache, caches):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


class Call:
    """One call's inputs and what it gives alone with a workspace of its own."""

    def __init__(self, seed, kind, B=1, H=16, n=11, P=4000):
        g = torch.Generator().manual_seed(seed)
        self.kind, i32 = kind, torch.int32
        self.length = torch.tensor([P - 7 * b for b in range(B)], dtype=i32, device=DEV)
        if kind == "prefill":
            self.args = [torch.randn(s, generator=g).to(BF16).to(DEV) for s in
                         ((B, n, H, 192), (B, P + n, H, 128), (B, P + n, H, 128), (B, P + n, 64))]
            nbytes = rapid.rapid_latent_prefill_attn_workspace_size(B, n, H, P + n)
        else:
            self.args = [torch.randn((B, H, n, 576), generator=g).to(BF16).to(DEV),
                         _latent.make_cache((B, P + n), kind == "q8", g).to(DEV)]
            nbytes = rapid.rapid_latent_attn_workspace_size(
                B, H, n, P + n, rapid.RAPID_CACHE_LATENT_Q8 if kind == "q8" else rapid.RAPID_DTYPE_BF16)
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
        self.alone = self.run(workspace=self.workspace)
        torch.cuda.synchronize()

    def run(self, **kw):
        call = rapid.latent_prefill_attn if self.kind == "prefill" else rapid.latent_attn
        return call(*self.args, self.length, **kw)

    def check(self, got, what):
        for x, y in zip(got, self.alone):
            assert torch.equal(x, y), what


def _mix():
    return [Call(1, "bf16"), Call(2, "q8", B=3, H=40, n=3, P=900), Call(3, "prefill", H=4, n=70, P=2000),
            Call(4, "q8", n=1, P=300), Call(5, "prefill", B=2, H=2, n=300, P=100)]


def test_two_streams_take_turns_without_waiting():
    calls, streams, got = _mix(), [torch.cuda.Stream() for _ in range(2)], []
    for i in range(40):
        with torch.cuda.stream(streams[i % 2]):
            got.append((calls[i % len(calls)], calls[i % len(calls)].run()))
    other = torch.cuda.Stream()
    got += [(c, c.run(stream=other)) for c in calls]         # a stream that is not the current one
    torch.cuda.synchronize()
    for i, (c, x) in enumerate(got):
        c.check(x, i)


def test_threads_call_at_once():
    calls, bad = _mix(), []

    def work(k):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for i in range(12):
                    c = calls[(k + i) % len(calls)]
                    x = c.run()
                    torch.cuda.current_stream().synchronize()
                    c.check(x, (k, i))
        except Exception as e:      # noqa: BLE001
            bad.append(e)

    ts = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not bad, bad


def test_graphs_replay_side_by_side():
    calls = _mix()
    graphs = []
    for c in calls:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = c.run()
        graphs.append((gr, out))
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(3):
        for (gr, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    for c, (_, out) in zip(calls, graphs):
        c.check(out, c.kind)


def test_calls_back_to_back_share_a_workspace():
    # the second call's kernels start while the first call's finish
    a, b = Call(6, "bf16", H=64, n=3, P=700), Call(7, "bf16", H=64, n=3, P=699)
    ws = torch.empty(max(a.workspace.numel(), b.workspace.numel()), dtype=torch.uint8, device=DEV)
    got = [(c, c.run(workspace=ws)) for c in (a, b) * 10]
    torch.cuda.synchronize()
    for i, (c, x) in enumerate(got):
        c.check(x, i)
