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
