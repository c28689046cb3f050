"""The 8-bit cache's operators together, as a decode loop uses them (GPU; calls the C ABI
through the binding).

A prompt enters in chunks (append, seal), then verify steps run: append the nodes' rows behind
the tail, attention on every layer, acceptance, commit of the accepted path in the tail, advance
of the tail, sealing of full blocks.  Every number a step needs is in device memory, so the same
step captured once in a CUDA graph and replayed has to give the eager loop's bits.  Every
attention output is compared with the 64-bit form on the caches as they stand, and the caches
with the 64-bit forms of append and seal.
"""
import numpy as np
import pytest
import torch

from long_context_speculative_gb300 import rapid
from long_context_speculative_gb300 import workloads as wl

import _q8

pytestmark = pytest.mark.gpu
DEV = "cuda"
B, HQ, HKV, D, NQ, LAYERS, V = 2, 8, 2, 128, 6, 2, 2000
CAP, MAX_PAGES, KEEP = 320, 20, 5
CHUNK = 150


def _rows(g, n, heads):
    return torch.randn((LAYERS, B, n, heads, D), generator=g).to(torch.bfloat16).to(DEV)


class Loop:
    def __init__(self):
        g = torch.Generator().manual_seed(3)
        z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device=DEV)   # noqa: E731
        self.K, self.V = z(LAYERS, B, HKV, CAP, D), z(LAYERS, B, HKV, CAP, D)
        n_pages = B * MAX_PAGES
        self.pages = z(LAYERS, n_pages, HKV, 2, 64, D, dtype=torch.float8_e4m3fn)
        self.scales = torch.ones((LAYERS, n_pages, HKV, 2), device=DEV)
        self.table = torch.randperm(n_pages, generator=g).to(torch.int32).view(B, MAX_PAGES).to(DEV)
        self.sealed, self.tail = z(B, dtype=torch.int32), z(B, dtype=torch.int32)
        self.inv_freq = (5e5 ** (-torch.arange(0, D, 2).double() / D)).float().to(DEV)
        self.qw = (1 + 0.1 * torch.randn(D, generator=g)).to(torch.bfloat16).to(DEV)
        self.kw = (1 + 0.1 * torch.randn(D, generator=g)).to(torch.bfloat16).to(DEV)
        self.q8 = rapid.Q8LayerTable(list(self.K), list(self.V), list(self.pages), list(self.scales))
        self.kv = rapid.KVLayerTable(list(self.K), list(self.V))

    def append(self, layer, x, out, row_offset=None):
        rapid.qkv_append(x[layer][:, :, :HQ], x[layer][:, :, HQ:HQ + HKV], x[layer][:, :, HQ + HKV:],
                         self.K[layer], self.V[layer], self.tail, self.inv_freq, self.qw, self.kw,
                         pos_offset=self.sealed, row_offset=row_offset, out=out)

    def seal(self):
        self.q8.seal(self.table, self.sealed, self.tail, KEEP)
        self.q8.seal_advance(self.table, self.sealed, self.tail, KEEP)

    def state(self):
        return [t.clone() for t in (self.K, self.V, self.pages.view(torch.uint8), self.scales,
                                    self.sealed, self.tail)]


def _prefill(loop, g):
    for n in (CHUNK, 41):
        x = _rows(g, n, HQ + 2 * HKV)
        out = torch.empty((B, HQ, n, D), dtype=torch.bfloat16, device=DEV)
        for layer in range(LAYERS):
            loop.append(layer, x, out)
        loop.tail += n
        loop.seal()


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
        steps.append(dict(x=_rows(g, NQ, HQ + 2 * HKV), depth=depth.to(DEV),
                          mask=torch.stack([wl.ancestor_mask(p) for p in parents]).to(DEV),
                          z=z.to(DEV), q=q.to(DEV), tok=tok.to(DEV), par=par.to(DEV)))
    return steps


def _attend(loop, s, Q, O, L):
    for layer in range(LAYERS):
        loop.append(layer, s["x"], Q[layer], s["depth"])
        rapid.verify_attn_q8(Q[layer], loop.K[layer], loop.V[layer], loop.pages[layer],
                             loop.scales[layer], loop.table, loop.sealed, loop.tail, s["mask"],
                             out=O[layer], lse=L[layer])


def _accept(loop, s, seed):
    res = rapid.accept(s["z"], s["q"], s["tok"], s["par"], seed=seed)
    loop.kv.commit(loop.tail, res["path"], res["n_accepted"])
    rapid.rapid_kv_advance(loop.tail, res["n_accepted"], NQ, CAP)
    loop.seal()
    return res


def _run_step(loop, s, Q, O, L, seed):
    _attend(loop, s, Q, O, L)
    return _accept(loop, s, seed)


def _buffers():
    Q = [torch.empty((B, HQ, NQ, D), dtype=torch.bfloat16, device=DEV) for _ in range(LAYERS)]
    L = [torch.empty((B, HQ, NQ), device=DEV) for _ in range(LAYERS)]
    return Q, [torch.empty_like(q) for q in Q], L


@pytest.mark.parametrize("tree", [False, True])
def test_decode_loop_against_the_64_bit_forms(tree):
    g = torch.Generator().manual_seed(4)
    loop = Loop()
    _prefill(loop, g)
    assert loop.sealed.tolist() == [128, 128] and loop.tail.tolist() == [63, 63]
    Q, O, L = _buffers()
    sealed_once = False
    for k, s in enumerate(_steps(g, 6, tree)):
        before = loop.state()
        _attend(loop, s, Q, O, L)
        K1, V1 = loop.K.cpu(), loop.V.cpu()                # with the step's rows
        res = _accept(loop, s, torch.tensor([77 + k], dtype=torch.int64, device=DEV))
        torch.cuda.synchronize()
        assert rapid.rapid_device_error(True) == 0
        K0, V0, pages0, scales0, sealed0, tail0 = [t.cpu() for t in before]
        pages0 = pages0.view(torch.float8_e4m3fn)
        for layer in range(LAYERS):
            x = s["x"][layer].cpu()
            q64, K, Vv, eq, ek = _q8.append(
                x[:, :, :HQ], x[:, :, HQ:HQ + HKV], x[:, :, HQ + HKV:], K0[layer], V0[layer],
                Q[layer].cpu(), tail0, loop.inv_freq.cpu(), loop.qw.cpu(), loop.kw.cpu(),
                pos_offset=sealed0, row_offset=s["depth"].cpu())
            _q8.check(Q[layer], q64, eq, "Q")
            _q8.check(K1[layer], K, ek, "K")
            assert torch.equal(V1[layer].double(), Vv)
            ref = _q8.attn(Q[layer].cpu(), K1[layer], V1[layer], pages0[layer], scales0[layer],
                           loop.table.cpu(), sealed0, tail0, s["mask"].cpu())
            _q8.check(O[layer], ref[0], ref[2], "O")
            _q8.check(L[layer], ref[1], ref[3], "LSE")
        # lengths: tail + 1 + accepted, then whole blocks over KEEP sealed
        n_acc = res["n_accepted"].cpu()
        grown = tail0 + 1 + n_acc
        blocks = (grown - KEEP).clamp(min=0) // 64
        sealed_once |= bool((blocks > 0).any())
        assert torch.equal(loop.tail.cpu(), grown - 64 * blocks)
        assert torch.equal(loop.sealed.cpu(), sealed0 + 64 * blocks)
        # what is sealed now is the 64-bit form of what the tail held
        for layer in range(LAYERS):
            for b in range(B):
                for j in range(int(blocks[b])):
                    page = int(loop.table[b, int(sealed0[b]) // 64 + j])
                    for g_ in range(HKV):
                        block = K0[layer][b, g_, 64 * j:64 * j + min(64, int(tail0[b]) - 64 * j)].double()
                        scale = float(loop.scales[layer, page, g_, 0])
                        code = loop.pages[layer, page, g_, 0].float().cpu().double()[:len(block)]
                        assert np.array_equal(_q8.e4m3_round((block / scale).numpy()), code.numpy())
    assert sealed_once


@pytest.mark.parametrize("tree", [False, True])
def test_captured_step_replays_like_eager_steps(tree):
    g = torch.Generator().manual_seed(5)
    eager, graph_loop = Loop(), Loop()
    _prefill(eager, torch.Generator().manual_seed(6))
    _prefill(graph_loop, torch.Generator().manual_seed(6))
    steps = _steps(g, 5, tree)
    Q, O, L = _buffers()
    want = []
    for k, s in enumerate(steps):
        res = _run_step(eager, s, Q, O, L, torch.tensor([k], dtype=torch.int64, device=DEV))
        torch.cuda.synchronize()
        want.append((eager.state(), [o.clone() for o in O], [x.clone() for x in L],
                     {k2: v.clone() for k2, v in res.items()}))
    held = {k: v.clone() for k, v in steps[0].items()}
    seed = torch.zeros(1, dtype=torch.int64, device=DEV)
    Q, O, L = _buffers()
    start = graph_loop.state()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = _run_step(graph_loop, held, Q, O, L, seed)
    torch.cuda.synchronize()
    for x, y in zip(graph_loop.state(), start):            # capturing ran nothing
        assert torch.equal(x, y)
    for k, s in enumerate(steps):
        for name, t in s.items():
            held[name].copy_(t)
        seed.fill_(k)
        graph.replay()
        torch.cuda.synchronize()
        state, o, lse, r = want[k]
        for x, y in zip(graph_loop.state(), state):
            assert torch.equal(x, y), k
        for layer in range(LAYERS):
            assert torch.equal(O[layer], o[layer]) and torch.equal(L[layer], lse[layer]), (k, layer)
        for name in r:
            assert torch.equal(res[name], r[name]), (k, name)
    assert rapid.rapid_device_error(True) == 0


def test_an_empty_cache_takes_its_first_token():
    loop = Loop()
    g = torch.Generator().manual_seed(8)
    x = _rows(g, 1, HQ + 2 * HKV)
    Q = torch.empty((B, HQ, 1, D), dtype=torch.bfloat16, device=DEV)
    loop.append(0, x, Q)
    O, L = rapid.verify_attn_q8(Q, loop.K[0], loop.V[0], loop.pages[0], loop.scales[0], loop.table,
                                loop.sealed, loop.tail)
    torch.cuda.synchronize()
    # one key: the output is its value
    v = x[0][:, 0, HQ + HKV:].repeat_interleave(HQ // HKV, dim=1)
    assert torch.equal(O[:, :, 0], v)
    score = (Q[:, :, 0].double() * loop.K[0][:, :, 0].repeat_interleave(HQ // HKV, dim=1).double()).sum(-1)
    assert float((L[:, :, 0].double() - score / D ** 0.5).abs().max()) < 1e-4
