"""Expanded attention of prompt chunks against the 64-bit form (GPU; calls the C ABI through the
binding)."""
import pytest
import torch

from long_context_speculative_gb300 import rapid

import _latent

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16
NAN, INF = float("nan"), float("inf")


@pytest.fixture(autouse=True)
def _no_error_bits():
    torch.cuda.synchronize()
    rapid.rapid_device_error(True)
    yield
    torch.cuda.synchronize()
    assert rapid.rapid_device_error(True) == 0


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _inputs(B, n, H, L, seed, packed=False):
    g = torch.Generator().manual_seed(seed)
    Q = torch.randn((B, n, H, 192), generator=g).to(BF16).to(DEV)
    kv = torch.randn((B, L, H, 256), generator=g).to(BF16).to(DEV)
    rows = torch.randn((B, L, 576), generator=g).to(BF16).to(DEV)
    K, V, R = kv[..., :128], kv[..., 128:], rows[..., 512:]
    if packed:
        K, V, R = K.contiguous(), V.contiguous(), R.contiguous()
    return Q, K, V, R


def _check(Q, K, V, R, prefix, counts=None, scale=_latent.SCALE):
    B, n, H, _ = Q.shape
    out = torch.full((B, n, H, 128), 7.0, dtype=BF16, device=DEV)
    lse = torch.full((B, H, n), 7.0, device=DEV)
    O, L = rapid.latent_prefill_attn(Q, K, V, R, _ints(prefix), None if counts is None else _ints(counts),
                                     0.0 if scale == _latent.SCALE else scale, out=out, lse=lse)
    Oe, Le, eO, eL = _latent.prefill(Q, K, V, R, prefix, counts, scale)
    for b in range(B):
        m = n if counts is None else counts[b]
        err, lerr = (O[b, :m].double() - Oe[b, :m]).abs(), (L[b, :, :m].double() - Le[b, :, :m]).abs()
        assert (err <= eO[b, :m]).all(), (b, float((err / eO[b, :m]).max()))
        assert (lerr <= eL[b, :, :m]).all(), (b, float((lerr / eL[b, :, :m]).max()))
        assert (O[b, m:] == 7.0).all() and (L[b, :, m:] == 7.0).all()
    return O, L


@pytest.mark.parametrize("B,n,H,prefix", [
    (1, 1, 1, [0]), (1, 1, 3, [127]), (1, 1, 2, [128]), (1, 2, 2, [511]), (1, 127, 2, [0]), (1, 128, 1, [0]),
    (1, 129, 2, [0]), (1, 256, 1, [1]), (1, 257, 2, [0]), (1, 300, 3, [200]), (2, 77, 3, [5, 300]),
    (2, 5, 2, [0, 1500]), (3, 140, 2, [0, 63, 1000]), (1, 600, 1, [55]), (1, 16, 4, [5000]), (1, 1030, 2, [0])])
def test_prefill(B, n, H, prefix):
    _check(*_inputs(B, n, H, max(prefix) + n + 3, seed=n + H), prefix)


@pytest.mark.parametrize("n,H,prefix,counts", [
    (300, 2, [0, 700, 40], [300, 1, 0]), (130, 3, [0, 0, 2000], [129, 128, 130]), (64, 160, [0, 0, 100], [64, 3, 10]),
    (300, 60, [0, 900, 100], [257, 300, 13])])
def test_prefill_ragged(n, H, prefix, counts):
    # also more blocks than SMs, and up to twice as many
    _check(*_inputs(3, n, H, max(p + c for p, c in zip(prefix, counts)), seed=n), prefix, counts)


def test_prefill_layouts():
    B, n, H, L = 2, 40, 3, 90
    Q, K, V, R = _inputs(B, n, H, L, seed=1)
    want = _check(Q, K, V, R, [50, 3])
    def heads_first(x):      # [B, H, rows, d] storage
        return x.transpose(1, 2).contiguous().transpose(1, 2)
    wide = torch.zeros((B, n, H, 256), dtype=BF16, device=DEV)
    wide[..., 64:] = Q
    for args in ((Q, K.contiguous(), V.contiguous(), R.contiguous()),
                 (heads_first(Q), heads_first(K), heads_first(V), R), (wide[..., 64:], K, V, R)):
        got = rapid.latent_prefill_attn(*args, _ints([50, 3]))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(rapid.RapidError):     # rows that repeat
        rapid.latent_prefill_attn(Q, K[:, :, :1].expand(-1, -1, H, -1), V, R, _ints([50, 3]))
    with pytest.raises(rapid.RapidError):
        rapid.latent_prefill_attn(Q, K, V[:, :50], R, _ints([50, 3]))


@pytest.mark.parametrize("prefix", [0, 300])
def test_prefill_scores_that_keep_rising(prefix):
    Q, K, V, R = _inputs(1, 400, 2, prefix + 400, seed=2)
    Q[:, ::3] *= 0.01
    for scale in (0.5, 4.0):
        _check(Q, K, V, R, [prefix], scale=scale)


@pytest.mark.parametrize("n,H,prefix", [(5, 2, 0), (300, 2, 0), (300, 2, 1000), (200, 3, 129), (520, 20, 0)])
def test_prefill_hidden_keys_and_other_queries_may_hold_anything(n, H, prefix):
    L = prefix + n + 200
    Q, K, V, R = _inputs(1, n, H, L, seed=n)
    clean = _check(Q, K, V, R, [prefix])
    at = n // 2                                            # token whose key and values are bad
    for x in (K, V):
        x[0, prefix + at, 0] = NAN                         # of head 0
        x[0, prefix + n:] = INF                            # behind the chunk
    V[0, prefix + n - 1, 1, 3] = -INF                      # the last token's value of head 1
    R[0, prefix + n:] = NAN
    Q[0, 1, 1] = NAN
    O, Ls = rapid.latent_prefill_attn(Q, K, V, R, _ints([prefix]))
    hit = torch.zeros((1, n, H), dtype=torch.bool, device=DEV)
    hit[0, at:, 0] = True
    hit[0, n - 1, 1] = True
    hit[0, 1, 1] = True
    assert torch.isnan(O[0, at:, 0]).all() and torch.isnan(Ls[0, 0, at:]).all() and torch.isnan(O[0, n - 1, 1]).any()
    assert torch.equal(O[~hit], clean[0][~hit])
    assert torch.equal(Ls.transpose(1, 2)[~hit], clean[1].transpose(1, 2)[~hit])


@pytest.mark.parametrize("H", [2, 400])
def test_prefill_leaves_sequences_alone_that_do_not_fit(H):
    Q, K, V, R = _inputs(4, 6, H, 600, seed=4, packed=True)
    prefix, counts = [595, -1, 20, 594], [6, 6, 7, 6]
    out = torch.full((4, 6, H, 128), 7.0, dtype=BF16, device=DEV)
    lse = torch.full((4, H, 6), 7.0, device=DEV)
    rapid.latent_prefill_attn(Q, K, V, R, _ints(prefix), _ints(counts), out=out, lse=lse)
    torch.cuda.synchronize()
    assert rapid.rapid_device_error(True) == 2
    assert (out[:3] == 7.0).all() and (lse[:3] == 7.0).all()
    want, _, eO, _ = _latent.prefill(Q[3:], K[3:], V[3:], R[3:], [594])
    assert ((out[3:].double() - want).abs() <= eO).all()
