"""Absorbed attention over 8-bit rows that rapid_latent_append did not write: any fp32 scales, e4m3
codes that are NaN (GPU; calls the C ABI through the binding).

The rows' values are those of rapid_latent_read, bf16(code * scale).  Over them the call is the
call over a bf16 cache: the same tiles, splits and products, so the same bits.
"""
import pytest
import torch

from long_context_speculative_gb300 import rapid

import _latent
from _latent import DC, DK, DR

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


def _same(a, b):
    """Equal values, NaN in the same places."""
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(nan=1.0), b.nan_to_num(nan=1.0))


def _rows(B, rows, g, scale):
    """8-bit rows with every code that is a number, and these scales [B, rows, 4]."""
    code = torch.randint(0, 255, (B, rows, DC), generator=g, dtype=torch.uint8)
    code[(code & 0x7f) == 0x7f] = 0x7e
    rope = torch.randn((B, rows, DR), generator=g).to(BF16)
    return _latent.pack(code.view(torch.float8_e4m3fn), rope, scale.float())


def _both(Q, cache, prefix, mask=None):
    """The call over 8-bit rows, and over the rows that rapid_latent_read makes of them."""
    rows = rapid.latent_read(cache, None, cache.shape[1])
    return rapid.latent_attn(Q, cache, _ints(prefix), mask), rapid.latent_attn(Q, rows, _ints(prefix), mask), rows


@pytest.mark.parametrize("H,n,prefix", [(16, 1, [700, 63]), (8, 4, [1, 500]), (32, 5, [300, 1000])])
@pytest.mark.parametrize("kind", ["one", "any", "signs"])
def test_scales_that_are_no_powers_of_two(H, n, prefix, kind):
    g = torch.Generator().manual_seed(H)
    cap = max(prefix) + n + 2
    # codes go up to 448: values of size 1
    s = torch.full((2, cap, 4), 2.0 ** -7 * (1 + 2.0 ** -7 - 2.0 ** -20)) if kind == "one" else \
        0.005 * torch.exp(torch.randn((2, cap, 4), generator=g))
    if kind == "signs":
        s *= torch.where(torch.rand(s.shape, generator=g) < 0.5, -1.0, 1.0)
    cache = _rows(2, cap, g, s).to(DEV)
    Q = torch.randn((2, H, n, DK), generator=g).to(BF16).to(DEV)
    (O, L), (Or, Lr), rows = _both(Q, cache, prefix)
    assert _same(O, Or) and _same(L, Lr)
    want, lse, eO, eL = _latent.attn(Q, rows, prefix)
    assert ((O.double() - want).abs() <= eO).all() and ((L.double() - lse).abs() <= eL).all()


def test_scales_and_codes_out_of_the_ordinary():
    g = torch.Generator().manual_seed(2)
    scales = [1.3, -1.0, -300.0, 0.0, -0.0, 1e-40, 2.0 ** -126, 2.0 ** 7, 2.0 ** 8, -2.0 ** 8, 1e30, 3e38, INF, -INF, NAN]
    codes = [0x7f, 0xff]
    B, P = len(scales) + len(codes) + 1, 130
    cache = _latent.make_cache((B, P + 1), True, g)
    for b, x in enumerate(scales):
        _latent.parts(cache)[2][b, 70, 1] = x
    for b, x in enumerate(codes):
        cache[len(scales) + b, 70, 200] = x
    cache = cache.to(DEV)
    Q = (torch.randn((B, 16, 1, DK), generator=g) / 8).to(BF16).to(DEV)
    (O, L), (Or, Lr), rows = _both(Q, cache, [P] * B)
    assert _same(O, Or) and _same(L, Lr)
    for b in range(B):
        bad = not bool(torch.isfinite(rows[b]).all())
        assert bool(torch.isnan(L[b]).all()) == bool(torch.isnan(Lr[b]).all())
        if b >= len(scales) and b < B - 1:       # NaN codes reach every query
            assert bad and torch.isnan(O[b]).all() and torch.isnan(L[b]).all()
    assert torch.isfinite(O[:2]).all() and torch.isfinite(O[-1]).all()


def test_every_code_with_every_kind_of_scale():
    # one row seen with all others hidden: O is the row
    g = torch.Generator().manual_seed(3)
    scales = [1.0, 0.0123, 2.0 ** -64, 2.0 ** 7, 2.0 ** 9, -3.7, 1e-39, 1.99]
    B = len(scales)
    code = torch.arange(256, dtype=torch.int32).repeat(2).to(torch.uint8)
    code = code[torch.randperm(512, generator=g)].expand(B, 1, DC).clone()
    rope = torch.zeros((B, 1, DR), dtype=BF16)
    s = torch.tensor(scales)[:, None, None].expand(B, 1, 4)
    Q = torch.zeros((B, 3, 1, DK), dtype=BF16, device=DEV)
    number = code.clone()
    number[(number & 0x7f) == 0x7f] = 0
    cache = _latent.pack(number.view(torch.float8_e4m3fn), rope, s).to(DEV)
    (O, L), _, rows = _both(Q, cache, [0] * B)
    assert torch.equal(O, rows[:, None, :, :DC].expand(-1, 3, -1, -1)) and (L == 0).all()
    # NaN codes: the score is NaN, and the row with it
    cache = _latent.pack(code.view(torch.float8_e4m3fn), rope, s).to(DEV)
    (O, L), (Or, Lr), _ = _both(Q, cache, [0] * B)
    assert torch.isnan(O).all() and torch.isnan(L).all() and torch.isnan(Or).all() and torch.isnan(Lr).all()


@pytest.mark.parametrize("n,prefix", [(5, [0, 59, 64]), (64, [0, 33, 70])])
def test_hidden_rows_may_have_nan_codes(n, prefix):
    g = torch.Generator().manual_seed(n)
    cache = _latent.make_cache((3, max(prefix) + n + 70), True, g).to(DEV)
    Q = torch.randn((3, 16, n, DK), generator=g).to(BF16).to(DEV)
    mask = (torch.rand((3, n, n), generator=g) < 0.5).to(torch.uint8).to(DEV)
    mask[:, :, 2] = 0                                     # a row of the step that nobody sees
    mask[:, :, 3] = 0
    mask[:, 1, 3] = 1                                     # one that one query sees
    clean = rapid.latent_attn(Q, cache, _ints(prefix), mask)
    x = cache.clone()
    for b, P in enumerate(prefix):
        x[b, P + 2:P + 4, 7] = 0x7f
        x[b, P + 3, 400] = 0xff
        x[b, P + n:, :DC] = 0x7f
    O, L = rapid.latent_attn(Q, x, _ints(prefix), mask)
    hit = torch.zeros_like(L, dtype=torch.bool)
    hit[:, :, 1] = True
    assert torch.isnan(O[hit]).all() and torch.isnan(L[hit]).all()
    assert torch.equal(O[~hit], clean[0][~hit]) and torch.equal(L[~hit], clean[1][~hit])
