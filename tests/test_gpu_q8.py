"""The 8-bit cache's operators against their 64-bit forms (GPU; calls the C ABI through the
binding): append with norm and rotation, sealing, attention.
"""
import numpy as np
import pytest
import torch

from long_context_speculative_gb300 import rapid
from long_context_speculative_gb300 import workloads as wl

import _q8

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _no_error_bits():
    torch.cuda.synchronize()
    rapid.rapid_device_error(True)
    yield
    torch.cuda.synchronize()
    assert rapid.rapid_device_error(True) == 0


def _to(x):
    return {k: v.to(DEV) if isinstance(v, torch.Tensor) else v for k, v in x.items()}


# ---------------------------------------------------------------------------
# Append
# ---------------------------------------------------------------------------

def _append_case(B, n, Hq, Hkv, d, dtype, rot, seed, norm=False, tree=False, ragged=None, base=0,
                 cap=None, fused=True):
    g = torch.Generator().manual_seed(seed)
    cap = n + 70 if cap is None else cap
    if fused:
        x = torch.randn((B, n, Hq + 2 * Hkv, d), generator=g).to(dtype)
        q, k, v = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
    else:
        x = None
        q, k, v = (torch.randn((B, n, H, d), generator=g).to(dtype) for H in (Hq, Hkv, Hkv))
    c = dict(K=torch.randn((B, Hkv, cap, d), generator=g).to(dtype),
             V=torch.randn((B, Hkv, cap, d), generator=g).to(dtype),
             prefix_len=torch.randint(0, cap - n + 1, (B,), generator=g, dtype=torch.int32),
             inv_freq=(10000.0 ** (-torch.arange(0, rot, 2).double() / max(rot, 1))).float() if rot else None)
    if norm:
        c["q_weight"] = (1 + 0.3 * torch.randn(d, generator=g)).to(dtype)
        c["k_weight"] = (1 + 0.3 * torch.randn(d, generator=g)).to(dtype)
    if base:
        c["pos_offset"] = torch.tensor([base + 977 * b for b in range(B)], dtype=torch.int32)
    if tree:
        depth = []
        for _ in range(B):
            par, dep = wl.random_tree(n, 6, g), [0] * n
            for i in range(1, n):
                dep[i] = dep[par[i]] + 1
            depth.append(dep)
        c["row_offset"] = torch.tensor(depth, dtype=torch.int32)
    if ragged is not None:
        c["n_rows"] = torch.tensor(ragged, dtype=torch.int32)
    return x, q, k, v, c


def _run_append(x, q, k, v, c, **kw):
    B, n, Hq, d = q.shape
    Q0 = torch.full((B, Hq, n, d), 7.0, dtype=q.dtype)
    ref = _q8.append(q, k, v, c["K"], c["V"], Q0, **{a: t for a, t in c.items() if a not in "KV"}, **kw)
    if x is not None:
        Hkv = k.shape[2]
        xd = x.to(DEV)
        qd, kd, vd = xd[:, :, :Hq], xd[:, :, Hq:Hq + Hkv], xd[:, :, Hq + Hkv:]
    else:
        qd, kd, vd = q.to(DEV), k.to(DEV), v.to(DEV)
    cd = _to(c)
    out = rapid.qkv_append(qd, kd, vd, cd["K"], cd["V"], cd["prefix_len"],
                           **{a: t for a, t in cd.items() if a not in ("K", "V", "prefix_len")},
                           out=Q0.to(DEV), **kw)
    torch.cuda.synchronize()
    _q8.check(out, ref[0], ref[3], "Q")
    _q8.check(cd["K"], ref[1], ref[4], "K")
    assert torch.equal(cd["V"].cpu().double(), ref[2])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,n,Hq,Hkv,d", [(1, 1, 32, 8, 128), (1, 11, 32, 8, 128), (4, 32, 28, 4, 128),
                                          (3, 5, 4, 1, 64), (2, 67, 14, 2, 64), (1, 3, 1, 1, 128)])
@pytest.mark.parametrize("norm", [False, True])
def test_append(dtype, B, n, Hq, Hkv, d, norm):
    _run_append(*_append_case(B, n, Hq, Hkv, d, dtype, d, seed=n + d, norm=norm, base=5000))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,rot", [(128, 0), (128, 16), (128, 48), (128, 112), (64, 16), (64, 32), (64, 48)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_partial_rotation(dtype, d, rot, interleaved):
    _run_append(*_append_case(2, 7, 6, 3, d, dtype, rot, seed=rot, norm=rot % 32 == 0, base=321),
                interleaved=interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
def test_append_tree_offsets_and_ragged_counts(interleaved):
    for dtype in (BF16, F32):
        _run_append(*_append_case(4, 9, 8, 2, 128, dtype, 128, seed=3, tree=True, ragged=[9, 0, 1, 5]),
                    interleaved=interleaved)


@pytest.mark.parametrize("base", [131072, 1 << 24, (1 << 31) - 1 - 5000])
def test_append_far_positions(base):
    _run_append(*_append_case(1, 3, 4, 2, 128, F32, 128, seed=9, base=base, fused=False))


def test_append_odd_frequencies():
    # above one radian per position, negative, zero, subnormal
    x, q, k, v, c = _append_case(1, 4, 2, 1, 64, F32, 32, seed=10, base=12345)
    c["inv_freq"] = torch.tensor([3.5, -0.25, 0.0, 1e-40, 6.2831855, 1e4, 1e-7, 0.5,
                                  1.0, 2.0, -3.0, 1e-3, 7e-5, 0.1, 0.2, 0.3])
    _run_append(x, q, k, v, c)


def test_append_long_chunk():
    x, q, k, v, c = _append_case(1, 700, 32, 8, 128, BF16, 128, seed=11, norm=True, base=40)
    _run_append(x, q, k, v, c)


@pytest.mark.parametrize("what", ["prefix", "negative", "count"])
def test_append_refuses_rows_that_do_not_fit(what):
    x, q, k, v, c = _append_case(3, 6, 4, 2, 64, BF16, 64, seed=12, cap=20)
    c["prefix_len"] = torch.tensor([3, 14, 0], dtype=torch.int32)
    if what == "prefix":
        c["prefix_len"][1] = 15
    elif what == "negative":
        c["prefix_len"][1] = -1
    else:
        c["n_rows"] = torch.tensor([6, 7, 2], dtype=torch.int32)
    _run_append(x, q, k, v, c)
    assert rapid.rapid_stream_status() == rapid.RAPID_EINVAL


# ---------------------------------------------------------------------------
# Seal
# ---------------------------------------------------------------------------

def _seal_case(layers, B, Hkv, cap, d, dtype, sealed, tails, seed, max_pages=12):
    g = torch.Generator().manual_seed(seed)
    n_pages = B * max_pages + 3
    size = torch.exp(2 * torch.randn((layers, B, Hkv, 1, d), generator=g))
    K = (torch.randn((layers, B, Hkv, cap, d), generator=g) * size).to(dtype)
    V = (torch.randn((layers, B, Hkv, cap, d), generator=g) / size).to(dtype)
    pages = torch.zeros((layers, n_pages, Hkv, 2, 64, d)).to(torch.float8_e4m3fn)
    scales = torch.full((layers, n_pages, Hkv, 2), 3.0)
    table = torch.randperm(n_pages, generator=g)[:B * max_pages].to(torch.int32).view(B, max_pages)
    return K, V, pages, scales, table.contiguous(), sealed, tails


def _run_seal(K, V, pages, scales, table, sealed, tails, keep):
    layers = K.shape[0]
    Kd, Vd, Pd, Sd = (t.to(DEV) for t in (K, V, pages, scales))
    sealed = torch.tensor(sealed, dtype=torch.int32)
    tails = torch.tensor(tails, dtype=torch.int32)
    td, sd, ld = table.to(DEV), sealed.to(DEV), tails.to(DEV)
    t = rapid.Q8LayerTable(list(Kd), list(Vd), list(Pd), list(Sd))
    t.seal(td, sd, ld, keep)
    torch.cuda.synchronize()
    assert torch.equal(sd.cpu(), sealed) and torch.equal(ld.cpu(), tails)
    t.seal_advance(td, sd, ld, keep)
    torch.cuda.synchronize()
    bad = False
    for layer in range(layers):
        k, v, pg, sc = (x[layer].double().numpy().copy() for x in (K, V, pages, scales))
        s2, l2, bad = _q8.seal(k, v, pg, sc, table.numpy(), sealed.numpy(), tails.numpy(), keep)
        assert np.array_equal(Kd[layer].cpu().double().numpy(), k, equal_nan=True)
        assert np.array_equal(Vd[layer].cpu().double().numpy(), v, equal_nan=True)
        assert np.array_equal(Sd[layer].cpu().double().numpy(), sc)
        assert np.array_equal(Pd[layer].cpu().double().numpy(), pg, equal_nan=True)
        assert np.array_equal(sd.cpu().numpy(), s2) and np.array_equal(ld.cpu().numpy(), l2)
    return bad


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("keep", [0, 1, 64, 130])
def test_seal(dtype, d, keep):
    case = _seal_case(2, 6, 2, 400, d, dtype, [0, 64, 192, 0, 128, 0], [0, 63, 64, 200, 321, 400],
                      seed=d + keep)
    assert not _run_seal(*case, keep)


def test_seal_many_heads_one_part():
    # more heads than the launch gives several parts to: part 0 alone seals and moves
    case = _seal_case(24, 8, 8, 208, 64, BF16, [64 * b for b in range(8)], [26 * b + 15 for b in range(8)],
                      seed=5)
    assert not _run_seal(*case, 0)


def test_seal_many_blocks():
    case = _seal_case(1, 1, 1, 2131, 128, BF16, [64], [2131], seed=6, max_pages=40)
    assert not _run_seal(*case, 11)


def test_seal_extreme_values():
    K, V, pages, scales, table, sealed, tails = _seal_case(1, 1, 2, 400, 64, F32, [0], [384], seed=7)
    V[0, 0, 0, :64] = 0                                    # an all-zero block
    V[0, 0, 0, 64:128] *= 1e-30                            # below the exponent's floor
    V[0, 0, 0, 128:192, 3] = float("inf")
    V[0, 0, 0, 130, 5] = float("nan")
    V[0, 0, 0, 192:256] = float("-inf")                    # nothing finite
    V[0, 0, 1, :64] = 448.0                                # exactly the largest code
    V[0, 0, 1, 64:128] = torch.linspace(-1, 1, 64 * 64).view(64, 64) * 2.0 ** 127
    V[0, 0, 1, 128:192] = 1e-42                            # subnormal
    K[0, 0, 0, :64] = torch.arange(-2048, 2048).view(64, 64) / 16.0    # ties
    K[0, 0, 1, 64, 0] = 448.0 * 2 ** 5 * (1 + 2.0 ** -20)  # just above a power of two times 448
    K[0, 0, 1, 65:128] = 0.01
    assert not _run_seal(K, V, pages, scales, table, sealed, tails, 0)


@pytest.mark.parametrize("what", ["tail", "tail_negative", "sealed", "sealed_negative", "table", "page",
                                  "page_negative"])
def test_seal_refuses_a_sequence(what):
    K, V, pages, scales, table, sealed, tails = _seal_case(2, 3, 2, 256, 64, BF16, [0, 64, 128],
                                                           [130, 200, 70], seed=8)
    if what == "tail":
        tails[1] = 257
    elif what == "tail_negative":
        tails[1] = -1
    elif what == "sealed":
        sealed[1] = 65
    elif what == "sealed_negative":
        sealed[1] = -64
    elif what == "table":
        sealed[1] = 64 * 10
    elif what == "page":
        table[1, 2] = pages.shape[1]
    else:
        table[1, 3] = -1
    assert _run_seal(K, V, pages, scales, table, sealed, tails, 0)
    assert rapid.rapid_stream_status() == rapid.RAPID_EINVAL


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------

def _run_attn(c, Q, mask=None, softmax_scale=0.0, ref=None):
    cd = _to(c)
    O, L = rapid.verify_attn_q8(Q.to(DEV), cd["K"], cd["V"], cd["pages"], cd["scales"],
                                cd["page_table"], cd["sealed_len"], cd["tail_len"],
                                None if mask is None else mask.to(DEV), softmax_scale)
    torch.cuda.synchronize()
    if ref is None:
        ref = _q8.attn(Q, c["K"], c["V"], c["pages"], c["scales"], c["page_table"], c["sealed_len"],
                       c["tail_len"], mask, softmax_scale or None)
    _q8.check(O, ref[0], ref[2], "O")
    _q8.check(L, ref[1], ref[3], "LSE")
    return O, L


def _queries(B, Hq, n, d, dtype, seed, size=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((B, Hq, n, d), generator=g) * size).to(dtype)


def _tree_masks(B, n, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.stack([wl.ancestor_mask(wl.random_tree(n, 6, g)) for _ in range(B)])


SHAPES = [  # Hq, Hkv, n_q: one row to a KV head, few, 44, 64, 65, 88, 128, 129, 224, 320
    (1, 1, 1), (4, 1, 1), (32, 8, 1), (4, 1, 5), (8, 2, 11), (8, 2, 16), (5, 1, 13), (8, 1, 11), (4, 2, 64),
    (3, 1, 43), (7, 1, 32), (10, 2, 64)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,n", SHAPES)
def test_attn_group_shapes(dtype, d, Hq, Hkv, n):
    c = _q8.cache(2, Hkv, d, dtype, [7, 2], [5, 63], n, seed=Hq + n)
    _run_attn(c, _queries(2, Hq, n, d, dtype, seed=n))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("blocks,tails", [([0], [0]), ([0], [1]), ([1], [0]), ([2], [0]), ([3], [127]),
                                          ([0], [128]), ([5], [300]), ([0, 9, 1], [64, 0, 17]),
                                          ([40, 0, 3, 3, 21], [0, 130, 1, 60, 12])])
def test_attn_lengths(dtype, blocks, tails):
    for n in (1, 6):
        c = _q8.cache(len(blocks), 2, 128, dtype, blocks, tails, n, seed=len(blocks) + n)
        _run_attn(c, _queries(len(blocks), 8, n, 128, dtype, seed=n))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attn_tree_mask_and_scale(dtype):
    c = _q8.cache(3, 2, 128, dtype, [4, 1, 6], [10, 100, 0], 32, seed=4, scale_spread=6)
    Q = _queries(3, 14, 32, 128, dtype, seed=5)
    _run_attn(c, Q, _tree_masks(3, 32, 6))
    _run_attn(c, Q, _tree_masks(3, 32, 7).bool(), softmax_scale=0.031)


def test_attn_large_batch():
    B = 70
    c = _q8.cache(B, 1, 64, BF16, [b % 5 for b in range(B)], [(7 * b) % 66 for b in range(B)], 2, seed=8)
    _run_attn(c, _queries(B, 2, 2, 64, BF16, seed=9))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,n", [(1, 7), (1, 20), (1, 43), (1, 60), (2, 44), (2, 60), (3, 50)])
def test_attn_many_tiles_to_a_block(d, G, n):
    # so many KV heads that every block takes a whole sequence: 13 to 15 tiles one after the
    # other at every number of rows a block can have, an odd number of pages at the end
    Hkv = 152
    c = _q8.cache(1, 2, d, BF16, [25], [150], n, seed=G + n, scale_spread=2)
    c["scales"][c["page_table"][0, 20].long(), :, 0] *= 64   # a late block whose keys outweigh the rest
    Q = _queries(1, 2 * G, n, d, BF16, seed=n)
    ref = _q8.attn(Q, c["K"], c["V"], c["pages"], c["scales"], c["page_table"], c["sealed_len"],
                   c["tail_len"])
    rep = Hkv // 2
    wide = dict(c, K=c["K"].repeat(1, rep, 1, 1), V=c["V"].repeat(1, rep, 1, 1),
                pages=c["pages"].view(torch.uint8).repeat(1, rep, 1, 1, 1).view(torch.float8_e4m3fn),
                scales=c["scales"].repeat(1, rep, 1).contiguous())
    ref = [x.repeat(1, rep, *([1] * (x.dim() - 2))) for x in ref]
    _run_attn(wide, Q.repeat(1, rep, 1, 1), ref=ref)


@pytest.mark.parametrize("B,Hkv", [(20, 8), (38, 8), (41, 16)])
def test_attn_more_sequences_than_fit_on_the_machine_at_once(B, Hkv):
    # more blocks than SMs even with one to a sequence; several splits of some, none of others
    blocks = [(5 * b) % 13 for b in range(B)]
    c = _q8.cache(B, Hkv, 64, BF16, blocks, [(7 * b) % 60 for b in range(B)], 1, seed=40)
    _run_attn(c, _queries(B, 2 * Hkv, 1, 64, BF16, seed=41))


def test_attn_more_row_blocks_than_sms():
    # one sequence whose heads and blocks of rows alone are more than the SMs
    c = _q8.cache(1, 40, 64, BF16, [9], [33], 64, seed=42)
    _run_attn(c, _queries(1, 320, 64, 64, BF16, seed=43))


def test_attn_long_history():
    c = _q8.cache(1, 1, 128, BF16, [300], [37], 11, seed=10, scale_spread=2)
    _run_attn(c, _queries(1, 4, 11, 128, BF16, seed=11))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("size", [1e-3, 8.0, 60.0])
def test_attn_query_sizes(dtype, size):
    # flat and very peaked softmax rows; the running maximum moves by many powers of two
    c = _q8.cache(1, 2, 128, dtype, [12], [40], 4, seed=12)
    _run_attn(c, _queries(1, 8, 4, 128, dtype, seed=13, size=size))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attn_rows_of_very_different_sizes(dtype):
    Q = _queries(1, 8, 4, 128, dtype, seed=14)
    Q[:, ::2] *= 2.0 ** -20
    Q[:, :, 1] *= 2.0 ** 6
    Q[:, 3, 2] = 0
    _run_attn(_q8.cache(1, 2, 128, dtype, [6], [40], 4, seed=15), Q)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attn_rising_scores(dtype):
    # every block's keys outweigh all earlier ones: the running maximum rises at each
    c = _q8.cache(1, 1, 128, dtype, [14], [70], 3, seed=16)
    Q = _queries(1, 4, 3, 128, dtype, seed=17).abs()
    c["pages"] = c["pages"].float().abs().to(torch.float8_e4m3fn)
    c["K"] = c["K"].abs()
    order = c["page_table"][0, :14].long()
    c["scales"][order, :, 0] = (2.0 ** (torch.arange(14) - 9.0))[:, None]
    _run_attn(c, Q)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attn_rows_without_a_visible_key(dtype):
    n = 5
    mask = torch.zeros((2, n, n), dtype=torch.uint8)
    mask[0, 0, 0] = 1
    mask[0, 3, 1] = 1
    c = _q8.cache(2, 1, 128, dtype, [0, 0], [0, 0], n, seed=18)
    O, L = _run_attn(c, _queries(2, 4, n, 128, dtype, seed=19), mask)
    assert torch.equal(O[1].cpu(), torch.zeros_like(O[1].cpu())) and (L[1] == -float("inf")).all()
    c = _q8.cache(2, 1, 128, dtype, [2, 0], [0, 3], n, seed=20)
    _run_attn(c, _queries(2, 4, n, 128, dtype, seed=21), mask)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_attn_hidden_rows_may_hold_anything(dtype, bad):
    # speculative rows that a query's mask hides, rows behind the last one, unused pages
    B, n, d = 2, 6, 128
    c = _q8.cache(B, 2, d, dtype, [3, 0], [9, 0], n, seed=22)
    mask = torch.eye(n, dtype=torch.uint8).repeat(B, 1, 1)
    mask[:, :, 0] = 1
    mask[:, 3] = torch.tensor([1, 0, 0, 0, 0, 0])
    Q = _queries(B, 8, n, d, dtype, seed=23)
    ref = _q8.attn(Q, c["K"], c["V"], c["pages"], c["scales"], c["page_table"], c["sealed_len"],
                   c["tail_len"], mask)
    for b in range(B):
        t = int(c["tail_len"][b])
        for x in (c["K"], c["V"]):
            x[b, :, t + 3] = bad                           # hidden from every query
            x[b, :, t + n:] = bad                          # behind the last row
            x[b, :, t + 4] = bad                           # seen by query 4 alone
    used = set(c["page_table"][0, :3].tolist())
    for i in range(c["pages"].shape[0]):
        if i not in used:
            c["pages"][i] = torch.tensor(float("nan")).to(torch.float8_e4m3fn)
            c["scales"][i] = bad
    cd = _to(c)
    O, L = rapid.verify_attn_q8(Q.to(DEV), cd["K"], cd["V"], cd["pages"], cd["scales"],
                                cd["page_table"], cd["sealed_len"], cd["tail_len"], mask.to(DEV))
    torch.cuda.synchronize()
    clean = [0, 1, 2, 3, 5]
    _q8.check(O[:, :, clean], ref[0][:, :, clean], ref[2][:, :, clean], "O")
    _q8.check(L[:, :, clean], ref[1][:, :, clean], ref[3][:, :, clean], "LSE")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("where", ["tail", "spec", "page"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_attn_visible_values_that_are_not_finite(dtype, where, bad):
    B, n, d = 1, 4, 128
    c = _q8.cache(B, 1, d, dtype, [4], [20], n, seed=24)
    if where == "tail":
        c["V"][0, 0, 3, 17] = bad
    elif where == "spec":
        c["V"][0, 0, 22, 17] = bad                         # node 2: queries 2 and 3 see it
    else:
        c["pages"][int(c["page_table"][0, 1]), 0, 1, 5, 17] = float("nan")
    _run_attn(c, _queries(B, 4, n, d, dtype, seed=25))


def test_attn_nan_query_stays_in_its_row():
    for dtype in (BF16, F32):
        c = _q8.cache(1, 1, 128, dtype, [3], [20], 4, seed=26)
        Q = _queries(1, 4, 4, 128, dtype, seed=27)
        ref = _q8.attn(Q, c["K"], c["V"], c["pages"], c["scales"], c["page_table"], c["sealed_len"],
                       c["tail_len"])
        Q[0, 2, 1, 5] = float("nan")
        cd = _to(c)
        O, L = rapid.verify_attn_q8(Q.to(DEV), cd["K"], cd["V"], cd["pages"], cd["scales"],
                                    cd["page_table"], cd["sealed_len"], cd["tail_len"])
        torch.cuda.synchronize()
        assert torch.isnan(O[0, 2, 1]).all()
        ref[0][0, 2, 1] = float("nan")
        ref[1][0, 2, 1] = L[0, 2, 1].cpu().double()
        _q8.check(O, ref[0], ref[2], "O")
        _q8.check(L, ref[1], ref[3], "LSE")


@pytest.mark.parametrize("what", ["sealed_odd", "sealed_long", "sealed_negative", "tail_long",
                                  "tail_negative", "page", "page_negative"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attn_flags_inputs_out_of_range(dtype, what):
    c = _q8.cache(3, 1, 64, dtype, [2, 3, 1], [7, 9, 11], 4, seed=28)
    Q = _queries(3, 2, 4, 64, dtype, seed=29)
    if what == "sealed_odd":
        c["sealed_len"][1] = 64 * 3 + 5
    elif what == "sealed_long":
        c["sealed_len"][1] = 64 * (c["page_table"].shape[1] + 1)
    elif what == "sealed_negative":
        c["sealed_len"][1] = -64
    elif what == "tail_long":
        c["tail_len"][1] = c["K"].shape[2] - 3
    elif what == "tail_negative":
        c["tail_len"][1] = -1
    else:
        c["page_table"][1, 0] = c["pages"].shape[0] if what == "page" else -7
    cd = _to(c)
    O, L = rapid.verify_attn_q8(Q.to(DEV), cd["K"], cd["V"], cd["pages"], cd["scales"],
                                cd["page_table"], cd["sealed_len"], cd["tail_len"])
    assert rapid.rapid_stream_status() == rapid.RAPID_EINVAL
    # the other sequences are not touched by it
    sel = {k: (v[[0, 2]] if k not in ("pages", "scales") else v) for k, v in c.items()}
    ref = _q8.attn(Q[[0, 2]], sel["K"], sel["V"], c["pages"], c["scales"], sel["page_table"],
                   sel["sealed_len"], sel["tail_len"])
    _q8.check(O[[0, 2]], ref[0], ref[2], "O")
    _q8.check(L[[0, 2]], ref[1], ref[3], "LSE")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attn_repeats_bit_for_bit_and_keeps_to_its_buffers(dtype):
    c = _q8.cache(3, 2, 128, dtype, [30, 4, 11], [7, 90, 0], 11, seed=30)
    cd, Q = _to(c), _queries(3, 8, 11, 128, dtype, seed=31).to(DEV)
    nbytes = rapid.rapid_verify_attn_q8_workspace_size(3, 8, 2, 128, 11, cd["K"].shape[2],
                                                       cd["page_table"].shape[1], rapid._dtype_code(Q))
    ws = torch.full((nbytes + 8192,), 0xA5, dtype=torch.uint8, device=DEV)
    out = torch.full((Q.numel() + 2048,), 3.0, dtype=dtype, device=DEV)
    lse = torch.full((3 * 8 * 11 + 2048,), 3.0, device=DEV)
    got = []
    for fill in (0xA5, 0xFF, 0x00):                        # the workspace needs no initialisation
        ws[4096:4096 + nbytes] = fill
        O = out[1024:1024 + Q.numel()].view(Q.shape)
        L = lse[1024:1024 + 3 * 8 * 11].view(3, 8, 11)
        rapid.rapid_verify_attn_q8(Q, cd["K"], cd["V"], cd["pages"], cd["scales"], cd["page_table"],
                                   cd["sealed_len"], cd["tail_len"], None, 0.0, O, L,
                                   ws[4096:4096 + nbytes])
        torch.cuda.synchronize()
        got.append((O.clone(), L.clone()))
    for O, L in got[1:]:
        assert torch.equal(O, got[0][0]) and torch.equal(L, got[0][1])
    assert (ws[:4096] == 0xA5).all() and (ws[4096 + nbytes:] == 0xA5).all()
    assert (out[:1024] == 3).all() and (out[1024 + Q.numel():] == 3).all()
    assert (lse[:1024] == 3).all() and (lse[1024 + 3 * 8 * 11:] == 3).all()


def test_attn_on_another_stream():
    c = _q8.cache(2, 2, 128, BF16, [20, 3], [7, 90], 11, seed=32)
    Q = _queries(2, 8, 11, 128, BF16, seed=33)
    cd, Qd = _to(c), Q.to(DEV)
    ref = rapid.verify_attn_q8(Qd, cd["K"], cd["V"], cd["pages"], cd["scales"], cd["page_table"],
                               cd["sealed_len"], cd["tail_len"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs = [rapid.verify_attn_q8(Qd, cd["K"], cd["V"], cd["pages"], cd["scales"], cd["page_table"],
                                 cd["sealed_len"], cd["tail_len"], stream=s) for _ in range(8)]
    torch.cuda.synchronize()
    for O, L in outs:
        assert torch.equal(O, ref[0]) and torch.equal(L, ref[1])
