"""Query rows of very different sizes in one call (GPU; calls the C ABI through the binding): a row
is computed from itself alone, whatever the rows beside it hold.  Rows of a padded batch are such
rows: rapid_qkv_append leaves what lies behind a sequence's count as it was.
"""
import pytest
import torch

from long_context_speculative_gb300 import rapid

import _q8

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
# rows of a KV head: one for every row count that the bf16 kernel is built for
GROUPS = [(1, 7), (1, 20), (1, 43), (1, 60), (2, 44), (2, 60)]


@pytest.fixture(autouse=True)
def _no_error_bits():
    torch.cuda.synchronize()
    rapid.rapid_device_error(True)
    yield
    torch.cuda.synchronize()
    assert rapid.rapid_device_error(True) == 0


def _attend(c, Q):
    d = {k: v.to(DEV) for k, v in c.items()}
    out = rapid.verify_attn_q8(Q.to(DEV), d["K"], d["V"], d["pages"], d["scales"], d["page_table"],
                               d["sealed_len"], d["tail_len"])
    torch.cuda.synchronize()
    return out


def _reference(c, Q):
    return _q8.attn(Q, c["K"], c["V"], c["pages"], c["scales"], c["page_table"], c["sealed_len"], c["tail_len"])


def _check_rows(got, ref, rows):
    """`rows`: truth values [B, Hq, n]."""
    _q8.check(got[0].cpu()[rows], ref[0][rows], ref[2][rows], "O")
    _q8.check(got[1].cpu()[rows], ref[1][rows], ref[3][rows], "LSE")


def _queries(Hq, n, d, dtype, seed, B=1):
    return torch.randn((B, Hq, n, d), generator=torch.Generator().manual_seed(seed)).to(dtype)


def _garbage(shape, dtype, seed):
    """Any bits: huge values, infinities and NaN among them."""
    g = torch.Generator().manual_seed(seed)
    if dtype == BF16:
        return torch.randint(-32768, 32768, shape, generator=g, dtype=torch.int32).to(torch.int16).view(BF16)
    return torch.randint(-2 ** 31, 2 ** 31 - 1, shape, generator=g, dtype=torch.int64).to(torch.int32).view(F32)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [2.0 ** 9, 2.0 ** 12, 2.0 ** 30, 2.0 ** 60, 3e38])
def test_a_huge_row_leaves_the_others_alone(dtype, d, size):
    c = _q8.cache(1, 2, d, dtype, [13], [40], 5, seed=d)
    Q = _queries(8, 5, d, dtype, seed=1)
    ref = _reference(c, Q)
    Q[0, 2, 1] = (torch.sign(Q[0, 2, 1].float()) * size).to(dtype)
    rows = torch.ones((1, 8, 5), dtype=torch.bool)
    rows[0, 2, 1] = False
    _check_rows(_attend(c, Q), ref, rows)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,n", GROUPS)
def test_rows_of_any_bits_at_every_row_count(d, G, n):
    # many tiles to a block, as if the rows from some node on were padding
    c = _q8.cache(1, 2, d, BF16, [25], [150], n, seed=G + n)
    c["scales"][c["page_table"][0, 20].long(), :, 0] *= 64
    Q = _queries(2 * G, n, d, BF16, seed=n)
    ref = _reference(c, Q)
    keep = n - n // 3
    Q[:, :, keep:] = _garbage((1, 2 * G, n - keep, d), BF16, seed=d)
    rep = 76
    wide = dict(c, K=c["K"].repeat(1, rep, 1, 1), V=c["V"].repeat(1, rep, 1, 1),
                pages=c["pages"].view(torch.uint8).repeat(1, rep, 1, 1, 1).view(torch.float8_e4m3fn),
                scales=c["scales"].repeat(1, rep, 1).contiguous())
    rows = torch.zeros((1, 2 * G * rep, n), dtype=torch.bool)
    rows[:, :, :keep] = True
    _check_rows(_attend(wide, Q.repeat(1, rep, 1, 1)),
                [x.repeat(1, rep, *([1] * (x.dim() - 2))) for x in ref], rows)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("log2_size", [-12, -20, -40, -80])
def test_small_rows_beside_a_large_one(dtype, log2_size):
    # keys so large that the small rows' scores are of order one
    c = _q8.cache(1, 2, 128, dtype, [6], [40], 4, seed=3)
    c["scales"][:, :, 0] *= 2.0 ** -log2_size
    c["K"] *= 2.0 ** -log2_size
    Q = _queries(8, 4, 128, dtype, seed=4)
    Q *= 2.0 ** log2_size
    Q[0, :, 2] *= 2.0 ** -log2_size
    rows = torch.ones((1, 8, 4), dtype=torch.bool)
    rows[0, :, 2] = False
    _check_rows(_attend(c, Q), _reference(c, Q), rows)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_vanishing_rows(dtype):
    c = _q8.cache(1, 2, 128, dtype, [6], [0], 3, seed=5)
    c["scales"][:, :, 0] *= 2.0 ** 119
    c["K"] *= 2.0 ** 114
    Q = _queries(8, 3, 128, dtype, seed=6) * 2.0 ** -112
    Q[0, 3, 1] = 0
    rows = torch.ones((1, 8, 3), dtype=torch.bool)
    _check_rows(_attend(c, Q), _reference(c, Q), rows)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_padded_batch_from_append_to_attention(dtype):
    B, Hq, Hkv, n, d = 3, 8, 2, 9, 128
    counts = [9, 1, 5]
    c = _q8.cache(B, Hkv, d, dtype, [7, 12, 0], [30, 3, 64], n, seed=7)
    x = _queries(n, Hq + 2 * Hkv, d, dtype, seed=8, B=B)
    Q = _garbage((B, Hq, n, d), dtype, seed=9).to(DEV)
    held = {k: v.to(DEV) for k, v in c.items()}
    xd = x.to(DEV)
    inv_freq = (10000.0 ** (-torch.arange(0, d, 2).double() / d)).float().to(DEV)
    rapid.qkv_append(xd[:, :, :Hq], xd[:, :, Hq:Hq + Hkv], xd[:, :, Hq + Hkv:], held["K"], held["V"],
                     held["tail_len"], inv_freq, pos_offset=held["sealed_len"],
                     n_rows=torch.tensor(counts, dtype=torch.int32, device=DEV), out=Q)
    got = rapid.verify_attn_q8(Q, held["K"], held["V"], held["pages"], held["scales"], held["page_table"],
                               held["sealed_len"], held["tail_len"])
    torch.cuda.synchronize()
    rows = torch.zeros((B, Hq, n), dtype=torch.bool)
    for b, m in enumerate(counts):
        rows[b, :, :m] = True
    Qc = torch.where(rows[..., None], Q.cpu(), torch.zeros((), dtype=dtype))
    ref = _reference(dict(c, K=held["K"].cpu(), V=held["V"].cpu()), Qc)
    _check_rows(got, ref, rows)
