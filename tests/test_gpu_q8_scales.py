"""Attention over pages whose V scales lie far apart (GPU; calls the C ABI through the binding).

A page counts by its probabilities and its values, whatever the scales of the pages beside it:
the errors here are bounded by the sum of p |v| of every output element alone, with no term in
the largest value of the history.
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


def _abs_codes(codes):
    return (codes.view(torch.uint8) & 0x7f).view(codes.dtype)


def _reference(c, Q, p_round, v_round):
    """O, LSE and the bounds of their errors.  Relative to p |v| of one key: the score's error ds
    and the sums' (both inside eL, which _q8.attn derives) count twice, through p and through the
    sum that p is divided by; then p's rounding and v's.  A probability is held as a power of two
    in fp32's normal range, the row's largest at 1 or more, so a key below 2^-126 of it may count
    as nothing: 2^-126 max|v| for each of N keys (the sum that p is divided by is 1 or more)."""
    at = [c[k] for k in ("page_table", "sealed_len", "tail_len")]
    O, L, _, eL = _q8.attn(Q, c["K"], c["V"], c["pages"], c["scales"], *at)
    pages = c["pages"].clone()
    pages[:, :, 1] = _abs_codes(pages[:, :, 1].contiguous())
    A = _q8.attn(Q, c["K"], c["V"].abs(), pages, c["scales"], *at)[0]
    used = c["page_table"][0, :int(c["sealed_len"][0]) // 64].long()
    big = pages[:, :, 1].float()[used].abs().double() * c["scales"][used, :, 1].double()[..., None, None]
    rows = c["V"][0, :, :int(c["tail_len"][0]) + Q.shape[2]].double().abs()
    lost = (64 * len(used) + rows.shape[1]) * 2.0 ** -126 * max(float(big.max()), float(rows.max()))
    e = A * (2 * eL[..., None] + p_round + v_round + p_round * v_round) + lost
    return O, L, e + _q8.HALF_STEP[Q.dtype] * (O.abs() + e), eL


def _run(c, Q, p_round, v_round=0.0, rep=1):
    """`rep`: that many copies of every KV head, so that one block takes many tiles."""
    O, L, eO, eL = _reference(c, Q, p_round, v_round)
    wide = dict(c)
    if rep > 1:
        wide["K"], wide["V"] = c["K"].repeat(1, rep, 1, 1), c["V"].repeat(1, rep, 1, 1)
        wide["pages"] = c["pages"].view(torch.uint8).repeat(1, rep, 1, 1, 1).view(c["pages"].dtype)
        wide["scales"] = c["scales"].repeat(1, rep, 1).contiguous()
        Q = Q.repeat(1, rep, 1, 1)
        O, L, eO, eL = (x.repeat(1, rep, *([1] * (x.dim() - 2))) for x in (O, L, eO, eL))
    d = {k: v.to(DEV) for k, v in wide.items()}
    got = rapid.verify_attn_q8(Q.to(DEV), d["K"], d["V"], d["pages"], d["scales"], d["page_table"],
                               d["sealed_len"], d["tail_len"])
    torch.cuda.synchronize()
    _q8.check(got[0], O, eO, "O")
    _q8.check(got[1], L, eL, "LSE")


def _case(dtype, d, blocks, tail, n, seed):
    c = _q8.cache(1, 2, d, dtype, [blocks], [tail], n, seed=seed)
    return c, c["page_table"][0, :blocks].long()


def _queries(Hq, n, d, dtype, seed):
    return torch.randn((1, Hq, n, d), generator=torch.Generator().manual_seed(seed)).to(dtype)


def _p(dtype):
    """Half a step of the coarsest type that probabilities are rounded to."""
    return 2.0 ** -8 if dtype == BF16 else 0.0


# ---------------------------------------------------------------------------
# Scales far apart
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rep", [1, 76])
def test_all_zero_blocks_beside_small_values(dtype, d, rep):
    # sealing gives an all-zero block scale 1: it adds nothing, and takes nothing from the others
    if dtype == F32 and rep > 1:
        rep = 4
    for small in (2.0 ** -16, 2.0 ** -28, 2.0 ** -64):
        c, order = _case(dtype, d, 13, 20, 5, seed=d)
        c["scales"][:, :, 1] = small
        c["V"] *= small
        for page in order[1::3].tolist():
            c["pages"][page, :, 1] = torch.zeros_like(c["pages"][page, :, 1].float()).to(c["pages"].dtype)
            c["scales"][page, :, 1] = 1.0
        _run(c, _queries(8, 5, d, dtype, seed=1), _p(dtype), rep=rep)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,n", GROUPS)
def test_all_zero_blocks_at_every_row_count(d, G, n):
    c, order = _case(BF16, d, 25, 150, n, seed=G + n)
    c["scales"][:, :, 1] = 2.0 ** -30
    c["V"] *= 2.0 ** -24
    for page in order[[3, 16, 24]].tolist():
        c["pages"][page, :, 1] = torch.zeros_like(c["pages"][page, :, 1].float()).to(c["pages"].dtype)
        c["scales"][page, :, 1] = 1.0
    c["scales"][order[20], :, 0] *= 64             # the references move late
    _run(c, _queries(2 * G, n, d, BF16, seed=n), _p(BF16), rep=76)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("log2_ratio", [14, 15, 16, 20, 24, 25, 30, 64, 110])
def test_small_pages_that_hold_the_probability(dtype, log2_ratio):
    # keys of the large pages point away from the queries: what is left of their probability is
    # far below the ratio of the scales
    for d in (64, 128):
        n = 5
        c, order = _case(dtype, d, 9, 0, n, seed=log2_ratio)
        codes = _abs_codes(c["pages"][:, :, 0].contiguous())
        c["scales"][:, :, 0] = 2.0 ** -4
        c["scales"][:, :, 1] = 2.0 ** -log2_ratio
        for page in order[[0, 3, 4, 7]].tolist():  # with a small page, with a large one, first
            codes[page] = (codes[page].view(torch.uint8) | 0x80).view(codes.dtype)
            c["scales"][page, :, 1] = 1.0
        c["pages"][:, :, 0] = codes
        c["K"] = -c["K"].abs()
        Q = _queries(8, n, d, dtype, seed=d).abs()
        _run(c, Q, _p(dtype))
        _run(c, Q, _p(dtype), rep=76 if dtype == BF16 else 2)


# ---------------------------------------------------------------------------
# Scales that are no powers of two
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("log2_ratio", [0, 3, 5, 6, 9, 14, 15, 20, 30])
def test_scales_that_are_no_powers_of_two(dtype, log2_ratio):
    # Values code * scale are rounded: twice to fp16 (2^-11 each) where no such scale of a block
    # lies further than 2^5 below its largest, else once to bf16 (2^-8) together with the
    # probabilities.  Equal codes in a dimension, down to e4m3's smallest: no rounding averages out.
    n, d = 3, 128
    near = log2_ratio <= 5
    p_round = 0.0 if dtype == F32 else 2.0 ** -11 if near else 2.0 ** -8
    v_round = 2.0 ** -24 if dtype == F32 else 2.0 ** -10 + 2.0 ** -22 if near else 2.0 ** -8
    for factor in (1.4, 4 / 3, 1.9990234, 1 + 2.0 ** -12):
        c, order = _case(dtype, d, 12, 0, n, seed=log2_ratio)
        c["scales"][:, :, 1] = factor * 2.0 ** -log2_ratio
        v = (2.0 ** -9 * torch.arange(1, d + 1) * torch.tensor([1.0, -1.0]).repeat(d // 2)).expand(64, d)
        v = v.to(c["pages"].dtype)
        c["pages"][:, :, 1] = v
        c["pages"][order[5], :, 1] = torch.zeros((64, d)).to(c["pages"].dtype)
        c["scales"][order[5], :, 1] = 1.0                  # the largest, with nothing in it
        if log2_ratio == 0:
            c["scales"][order[5], :, 1] = factor
        c["V"] *= 0                                        # the pages' roundings alone
        _run(c, _queries(8, n, d, dtype, seed=3), p_round, v_round)
        _run(c, _queries(8, n, d, dtype, seed=4), p_round, v_round, rep=76 if dtype == BF16 else 2)


# ---------------------------------------------------------------------------
# Scales far from one, beside tail rows
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("log2_scale", [-126, -110, -64, -33, -32, 32, 33, 64, 110, 119])
def test_tail_rows_beside_far_scales(dtype, log2_scale):
    # the tail's values are of order one; pages of a large scale hold zeros
    n, d = 4, 128
    c, order = _case(dtype, d, 5, 40, n, seed=7)
    c["scales"][:, :, 1] = 2.0 ** log2_scale
    if log2_scale > 0:
        c["pages"][:, :, 1] = torch.zeros(c["pages"][:, :, 1].shape).to(c["pages"].dtype)
    Q = _queries(8, n, d, dtype, seed=8) * 4      # probabilities of very different sizes
    _run(c, Q, _p(dtype))
    _run(c, Q, _p(dtype), rep=76 if dtype == BF16 else 2)
