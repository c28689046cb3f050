"""Guard bands around the outputs, caches and workspaces of the latent cache's calls (GPU; calls the
C ABI through the binding): what a call writes stands between bytes of a fill pattern, which have to
be there after it, and rows that it has no business with stay as they were.
"""
import pytest
import torch

from long_context_speculative_gb300 import rapid

import _latent
from test_gpu_canary import Guarded, _check

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, U8, F32, I32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32


def _ints(v):
    return torch.tensor(v, dtype=I32, device=DEV)


def _cache(B, cap, q8, g):
    x = _latent.make_cache((B, cap), q8, g).to(DEV)
    c = Guarded(tuple(x.shape), x.dtype)
    c.t.copy_(x)
    return c, x


INV = (5e5 ** (-torch.arange(0, 64, 2).double() / 64)).float()


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("n,H,counts", [(1, 1, None), (11, 128, None), (300, 9, [300, 1, 77])])
def test_append(q8, n, H, counts):
    g = torch.Generator().manual_seed(n)
    B, cap = 3, n + 5
    c, before = _cache(B, cap, q8, g)
    prefix = [5, 0, 3]                                    # up to the last row of the cache
    kv = torch.randn((B, n, 576), generator=g).to(BF16).to(DEV)
    q = torch.randn((B, n, H, 64), generator=g).to(BF16).to(DEV)
    out = Guarded((B, n, H, 64), BF16)
    for _ in range(2):
        rapid.latent_append(kv, c.t, _ints(prefix), INV.to(DEV), q=q, q_out=out.t,
                            n_rows=None if counts is None else _ints(counts))
    _check(("cache", c), ("q_out", out))
    for b in range(B):
        m = n if counts is None else counts[b]
        rest = torch.ones(cap, dtype=torch.bool)
        rest[prefix[b]:prefix[b] + m] = False
        assert torch.equal(c.t[b, rest.to(DEV)].view(U8), before[b, rest.to(DEV)].view(U8))


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("n", [1, 3, 67])
def test_read(q8, n):
    g = torch.Generator().manual_seed(n)
    _, x = _cache(3, n + 5, q8, g)
    rows = Guarded((3, n, 576), BF16)
    for _ in range(2):
        rapid.latent_read(x, _ints([5, 0, 2]), n, out=rows.t)
    _check(("rows", rows))


@pytest.mark.parametrize("q8", [False, True])
def test_commit(q8):
    g = torch.Generator().manual_seed(1)
    B, n_q, cap = 2, 64, 70
    layers = [_cache(B, cap, q8, g) for _ in range(3)]
    path = torch.full((B, n_q), -1, dtype=I32)
    path[0, :31] = torch.arange(2, 64, 2)
    path[1, :40] = torch.arange(24, 64)
    prefix, acc = [6, 0], [31, 40]                        # the last rows of the cache are among the sources
    table = rapid.LatentLayerTable([c.t for c, _ in layers])
    table.commit(_ints(prefix), path.to(DEV), _ints(acc))
    _check(*((f"cache {i}", c) for i, (c, _) in enumerate(layers)))
    for c, before in layers:
        for b in range(B):
            rest = torch.ones(cap, dtype=torch.bool, device=DEV)
            rest[prefix[b] + 1:prefix[b] + 1 + acc[b]] = False
            assert torch.equal(c.t[b, rest].view(U8), before[b, rest].view(U8))


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("B,H,n,prefix", [
    (1, 16, 1, [1000]), (1, 17, 1, [0]), (2, 5, 13, [900, 3]), (1, 128, 11, [5000]), (3, 3, 64, [10, 640, 63]),
    (33, 2, 3, None), (700, 1, 2, None)])
def test_attn(q8, B, H, n, prefix):
    g = torch.Generator().manual_seed(B + H)
    prefix = [(37 * b) % 401 for b in range(B)] if prefix is None else prefix
    cap = max(prefix) + n
    Q = torch.randn((B, H, n, 576), generator=g).to(BF16).to(DEV)
    c, before = _cache(B, cap, q8, g)
    O, L = Guarded((B, H, n, 512), BF16), Guarded((B, H, n), F32)
    ws = Guarded((rapid.rapid_latent_attn_workspace_size(
        B, H, n, cap, rapid.RAPID_CACHE_LATENT_Q8 if q8 else rapid.RAPID_DTYPE_BF16),), U8)
    for _ in range(2):
        rapid.latent_attn(Q, c.t, _ints(prefix), out=O.t, lse=L.t, workspace=ws.t)
    _check(("O", O), ("LSE", L), ("workspace", ws), ("cache", c))
    assert torch.equal(c.t.view(U8), before.view(U8))
    assert torch.isfinite(O.t.float()).all() and torch.isfinite(L.t).all()


@pytest.mark.parametrize("B,n,H,prefix,counts", [
    (1, 1, 1, [0], None), (1, 16, 4, [5000], None), (2, 300, 3, [0, 700], [1, 300]), (1, 257, 160, [0], None),
    (3, 130, 2, [511, 0, 40], [129, 0, 130]), (1, 520, 20, [900], None), (152, 3, 2, None, None)])
def test_prefill(B, n, H, prefix, counts):
    g = torch.Generator().manual_seed(n)
    prefix = [5 * b for b in range(B)] if prefix is None else prefix
    rows = max(p + (n if counts is None else counts[b]) for b, p in enumerate(prefix))
    Q, K, V, R = (torch.randn(s, generator=g).to(BF16).to(DEV) for s in
                  ((B, n, H, 192), (B, rows, H, 128), (B, rows, H, 128), (B, rows, 64)))
    O, L = Guarded((B, n, H, 128), BF16), Guarded((B, H, n), F32)
    O.t.fill_(7), L.t.fill_(7)
    ws = Guarded((rapid.rapid_latent_prefill_attn_workspace_size(B, n, H, rows),), U8)
    for _ in range(2):
        rapid.latent_prefill_attn(Q, K, V, R, _ints(prefix), None if counts is None else _ints(counts), out=O.t,
                                  lse=L.t, workspace=ws.t)
    _check(("O", O), ("LSE", L), ("workspace", ws))
    for b in range(B):
        m = n if counts is None else counts[b]
        assert (O.t[b, m:] == 7).all() and (L.t[b, :, m:] == 7).all()
        assert (O.t[b, :m].float() != 7).any(-1).all() and torch.isfinite(L.t[b, :, :m]).all()
