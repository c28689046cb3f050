"""Runs of several key tiles in one block of the latent attention kernels (GPU; calls the C ABI
through the binding).

With as many sequences as there is room for splits, every sequence is one split: all its tiles pass
through one block, round the rooms of shared memory several times.  The tests say from the
workspace's size that this is so.  A few sequences are compared with the 64-bit form and the others
are copies of them, whose results have to be the same bits.
"""
import math

import pytest
import torch

from long_context_speculative_gb300 import rapid

import _latent
from _latent import DK

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16
NAN, INF = float("nan"), float("inf")
TILE = 64


@pytest.fixture(autouse=True)
def _no_error_bits():
    torch.cuda.synchronize()
    rapid.rapid_device_error(True)
    yield
    torch.cuda.synchronize()
    assert rapid.rapid_device_error(True) == 0


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _up256(x):
    return (x + 255) // 256 * 256


def _slots(B, H, n, cap, q8):
    """Splits that a call has room for, from its workspace: parts of 512 values, a maximum and a sum for every
    row of a split, and two numbers a sequence; one split a sequence needs no parts."""
    nbytes = rapid.rapid_latent_attn_workspace_size(
        B, H, n, cap, rapid.RAPID_CACHE_LATENT_Q8 if q8 else rapid.RAPID_DTYPE_BF16)
    left = nbytes - 2 * _up256(4 * B)
    for S in range(B, 1000):
        rows = S * H * n if S > B else 0
        if _up256(rows * 2048) + _up256(rows * 8) == left:
            return S
    raise AssertionError(nbytes)


def _copies(x, B):
    """Sequences 0, 1, .., k - 1, 0, 1, .. up to B of them."""
    return x.repeat((B + x.shape[0] - 1) // x.shape[0], *(1,) * (x.dim() - 1))[:B].contiguous()


def _compare(Q, cache, prefix, B, mask=None):
    """The call on B copies of these sequences against the 64-bit form; O and LSE of the first ones."""
    k = len(prefix)
    O, L = rapid.latent_attn(_copies(Q, B), _copies(cache, B), _copies(_ints(prefix), B),
                             None if mask is None else _copies(mask, B))
    assert torch.equal(O, _copies(O[:k], B)) and torch.equal(L, _copies(L[:k], B))
    want, lse, eO, eL = _latent.attn(Q, cache, prefix, mask)
    O, L = O[:k], L[:k]
    empty = lse == -math.inf
    assert torch.equal(L == -math.inf, empty) and (O[empty] == 0).all()
    assert ((O.double() - want).abs() <= eO)[~empty].all(), float(((O.double() - want).abs() / eO)[~empty].max())
    assert ((L.double() - lse).abs() <= eL)[~empty].all()
    return O, L


SHAPES = [(16, 1, 700), (8, 4, 700), (32, 2, 700), (13, 5, 400)]     # 16, 32, 64 and 65 rows


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("H,n,B", SHAPES)
def test_attn_splits_of_one_to_six_tiles(q8, H, n, B):
    g = torch.Generator().manual_seed(H)
    prefix = [TILE * t - n - (t & 1) for t in range(1, 7)]
    Q = torch.randn((6, H, n, DK), generator=g).to(BF16).to(DEV)
    cache = _latent.make_cache((6, 6 * TILE + 7), q8, g).to(DEV)
    assert _slots(B, H, n, cache.shape[1], q8) == B
    _compare(Q, cache, prefix, B)


@pytest.mark.parametrize("H,prefix,counts", [(2, [0, 1, 130, 700], None), (80, [0, 300, 5, 700], [300, 1, 129, 64])])
def test_prefill_rings_of_any_fill(H, prefix, counts):
    # one to eight tiles of keys: fewer chunks than the ring has, as many, and more
    g = torch.Generator().manual_seed(H)
    n = 300
    L = max(prefix) + n
    Q, K, V, R = (torch.randn(s, generator=g).to(BF16).to(DEV) for s in
                  ((4, n, H, 192), (4, L, H, 128), (4, L, H, 128), (4, L, 64)))
    O, S = rapid.latent_prefill_attn(Q, K, V, R, _ints(prefix), None if counts is None else _ints(counts))
    heads = [0, H - 1]
    want, lse, eO, eL = _latent.prefill(Q[:, :, heads], K[:, :, heads], V[:, :, heads], R, prefix, counts)
    for b in range(4):
        m = n if counts is None else counts[b]
        assert ((O[b, :m, heads].double() - want[b, :m]).abs() <= eO[b, :m]).all()
        assert ((S[b, heads, :m].double() - lse[b, :, :m]).abs() <= eL[b, :, :m]).all()


def _rising(H, n, prefix, q8, g):
    """Queries and rows whose scores pass all before them by far more than 2^16 at tiles that differ from query
    to query (three in four of them), or fall, or stay."""
    k = len(prefix)
    Q = torch.randn((k, H, n, DK), generator=g)
    cap = max(prefix) + n + 3
    x = torch.randn((k, cap, DK), generator=g)
    tile = torch.arange(cap) // TILE
    x[..., 3] = 20.0 * tile                       # times 16 and 192^-0.5: 23 a tile
    x[..., 130] = 24.0 * (tile >= 2)
    x[..., 500] = 24.0 * (tile >= 3) + 24.0 * (tile >= 5)
    row = torch.arange(H * n).view(H, n)
    Q[..., 3] = torch.where(row % 4 == 0, 16.0, torch.where(row % 4 == 1, -16.0, 0.0))
    Q[..., 130] = torch.where(row % 3 == 0, 16.0, 0.0)
    Q[..., 500] = torch.where(row % 5 < 2, 16.0, 0.0)
    if not q8:
        cache = x.bfloat16()
    else:
        y = x[..., :512].unflatten(-1, (4, 128))
        s = _latent.group_scale(y.abs().amax(-1).double()).float()
        cache = _latent.pack((y / s[..., None]).flatten(-2).to(torch.float8_e4m3fn), x[..., 512:].bfloat16(), s)
    return Q.to(BF16).to(DEV), cache.to(DEV)


def _references_that_move(Q, cache, P, n):
    """How many of a query's tiles move its reference, by the scores themselves (most of any query)."""
    x = (Q[0].double().flatten(0, 1) @ _latent.values(cache[0, :P]).T) * _latent.SCALE / math.log(2)
    top = x[:, :P // TILE * TILE].unflatten(1, (-1, TILE)).amax(-1)
    ref, moved = top[:, 0].clone(), torch.zeros(top.shape[0], device=DEV)
    for t in range(1, top.shape[1]):
        up = top[:, t] > ref + 16
        moved += up
        ref = torch.where(up, top[:, t], ref)
    return moved


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("H,n,B", SHAPES)
def test_attn_references_move_from_tile_to_tile(q8, H, n, B):
    g = torch.Generator().manual_seed(H + 1)
    prefix = [6 * TILE - n, 450, 129, 320]
    Q, cache = _rising(H, n, prefix, q8, g)
    assert _slots(B, H, n, cache.shape[1], q8) == B
    moved = _references_that_move(Q, cache, prefix[0], n)
    assert moved.max() >= 4 and (moved == 0).any()
    _compare(Q, cache, prefix, B)


@pytest.mark.parametrize("q8", [False, True])
def test_attn_references_move_in_splits_of_several_tiles(q8):
    # few splits of many rows, joined: at least five tiles each
    g = torch.Generator().manual_seed(3)
    H, n, P = 128, 11, 2400
    Q, cache = _rising(H, n, [P], q8, g)
    S = _slots(1, H, n, cache.shape[1], q8)
    assert 1 < S and (P + n + TILE - 1) // TILE >= 5 * S, S
    assert _references_that_move(Q, cache, P, n).max() >= 4
    _compare(Q, cache, [P], 1)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("H,n,B", [(3, 5, 700), (6, 5, 700), (1, 64, 700), (13, 5, 400)])
def test_attn_hidden_rows_behind_several_tiles_may_hold_anything(q8, H, n, B):
    g = torch.Generator().manual_seed(n + H)
    prefix = [3 * TILE - 2, 4 * TILE, 2 * TILE + 33]
    Q = torch.randn((3, H, n, DK), generator=g).to(BF16).to(DEV)
    cache = _latent.make_cache((3, max(prefix) + n + 70), q8, g).to(DEV)
    assert _slots(B, H, n, cache.shape[1], q8) == B
    mask = (torch.rand((3, n, n), generator=g) < 0.5).to(torch.uint8).to(DEV)
    mask[:, :, 2] = 0                                     # rows of the step that nobody sees
    mask[:, :, 3] = 0
    mask[:, 1, 3] = 1                                     # one that one query sees
    clean_O, clean_L = _compare(Q, cache, prefix, B, mask)
    x = cache.clone()
    for b, P in enumerate(prefix):
        if q8:
            _latent.parts(x)[2][b, P + 2:P + 4] = NAN
            _latent.parts(x)[1][b, P + 2:P + 4] = INF
        else:
            x[b, P + 2:P + 4] = NAN
            x[b, P + 3, ::2] = INF
        x[b, P + n:] = 0xff if q8 else NAN                # behind the step
    O, L = rapid.latent_attn(_copies(Q, B), _copies(x, B), _copies(_ints(prefix), B), _copies(mask, B))
    assert torch.isnan(O[:, :, 1]).all() and torch.isnan(L[:, :, 1]).all()
    others = [i for i in range(n) if i != 1]
    assert torch.equal(O[:, :, others], _copies(clean_O[:, :, others], B))
    assert torch.equal(L[:, :, others], _copies(clean_L[:, :, others], B))


@pytest.mark.parametrize("n,H", [(1, 3), (300, 2), (100, 5)])
def test_prefill_references_move_in_runs_of_several_tiles(n, H):
    # blocks behind a long prefix, their keys shared out over all SMs: a run is several tiles of 128
    g = torch.Generator().manual_seed(n)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    blocks = (n + 255) // 256
    P = 128 * (4 * sms // (H * blocks) + 3)
    L = P + n
    Q = torch.randn((1, n, H, 192), generator=g)
    K = torch.randn((1, L, H, 128), generator=g)
    V = torch.randn((1, L, H, 128), generator=g).to(BF16).to(DEV)
    R = torch.randn((1, L, 64), generator=g).to(BF16).to(DEV)
    tile = torch.arange(L) // 128
    K[..., 3] = (20.0 * (tile % 5))[None, :, None]        # up by 23 a tile four times, and down
    K[..., 70] = (0.5 * tile)[None, :, None]
    Q[..., 3] = torch.where(torch.arange(n)[:, None] % 3 == 0, 16.0, 0.0)
    Q[..., 70] = torch.where(torch.arange(n)[:, None] % 4 == 1, 16.0, 0.0)
    Q, K = Q.to(BF16).to(DEV), K.to(BF16).to(DEV)
    # (parts of two slots an SM of 256 tokens, maxima and sums)
    assert rapid.rapid_latent_prefill_attn_workspace_size(1, n, H, L) > 2 * sms * 256 * 128 * 4
    O, S = rapid.latent_prefill_attn(Q, K, V, R, _ints([P]))
    want, lse, eO, eL = _latent.prefill(Q, K, V, R, [P])
    assert ((O.double() - want).abs() <= eO).all(), float(((O.double() - want).abs() / eO).max())
    assert ((S.double() - lse).abs() <= eL).all()


@pytest.mark.parametrize("B,H,n,P", [(3, 27, 1100, 0), (1, 130, 700, 40), (2, 11, 300, 12000), (1, 9, 9000, 0)])
def test_prefill_every_block_of_many_heads(B, H, n, P):
    # more blocks than the SMs share out by key tiles: heads are taken in groups, the last one larger
    g = torch.Generator().manual_seed(H)
    gd = torch.Generator(device=DEV).manual_seed(H)
    L = P + n
    Q, K, V, R = (torch.randn(s, generator=gd, device=DEV).to(BF16) for s in
                  ((B, n, H, 192), (B, L, H, 128), (B, L, H, 128), (B, L, 64)))
    O = torch.full((B, n, H, 128), 7.0, dtype=BF16, device=DEV)
    S = torch.full((B, H, n), 7.0, device=DEV)
    rapid.latent_prefill_attn(Q, K, V, R, _ints([P] * B), out=O, lse=S)
    assert (O != 7).any(-1).all() and (S != 7).all()
    heads = sorted({0, H // 2, H - 1, int(torch.randint(H, (1,), generator=g))})
    rows = torch.tensor(sorted({0, 1, 255, 256, n // 2, n - 2, n - 1} & set(range(n))), device=DEV)
    for b in range(B):
        for h in heads:
            k = torch.cat([K[b, :, h], R[b]], -1).double()
            x = (Q[b, rows, h].double() @ k.T * _latent.SCALE)
            hidden = torch.arange(L, device=DEV)[None] > P + rows[:, None]
            x = x.masked_fill(hidden, -math.inf)
            p, lse = _latent._softmax(x)
            mag = Q[b, rows, h].double().abs() @ k.abs().T * _latent.SCALE
            o = p @ V[b, :, h].double()
            eo, el = _latent._bounds(x, mag, p, V[b, :, h].double(), o, lse, L, 192 // 16 + 1)
            assert ((O[b, rows, h].double() - o).abs() <= eo).all() and ((S[b, h, rows].double() - lse).abs() <= el).all()
