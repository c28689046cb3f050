"""Latent cache: append, read back, commit and absorbed attention against 64-bit forms (GPU; calls
the C ABI through the binding)."""
import math

import pytest
import torch

from long_context_speculative_gb300 import rapid

import _latent
from _latent import DC, DK, DR, BF16_HALF

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16
NAN, INF = float("nan"), float("inf")
BAD_INPUT = 2


@pytest.fixture(autouse=True)
def _no_error_bits():
    torch.cuda.synchronize()
    rapid.rapid_device_error(True)
    yield
    torch.cuda.synchronize()
    assert rapid.rapid_device_error(True) == 0


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _gen(seed):
    return torch.Generator().manual_seed(seed)


# ---------------------------------------------------------------------------
# Append
# ---------------------------------------------------------------------------

def _inv_freq(g):
    f = 5e5 ** (-torch.arange(0, DR, 2).double() / DR)
    return f.float()


def _check_append(q8, B, n, H, prefix, cap, interleaved=False, weight=True, offsets=None, counts=None, eps=1e-6,
                  kv=None, seed=1, q_kind="strided"):
    g = _gen(seed)
    kv = torch.randn((B, n, DK), generator=g).mul(3).to(BF16) if kv is None else kv
    w = (1 + 0.2 * torch.randn(DC, generator=g)).to(BF16) if weight else None
    inv = _inv_freq(g)
    before = _latent.make_cache((B, cap), q8, g)
    cache = before.to(DEV)
    q = Q = q_out = None
    if H:
        # the rotated part of a projection's heads, into the last values of absorbed queries
        proj = torch.randn((B, n, H, 192), generator=g).to(BF16).to(DEV)
        Q = torch.randn((B, H, n, DK), generator=g).to(BF16).to(DEV)
        q = proj[..., 128:]
        q_out = {"strided": Q[..., DC:].transpose(1, 2), "in place": q, "new": None}[q_kind]
    q_before = q.clone() if H else None
    Q_before = Q.clone() if H else None
    # rows of a wider projection
    wide = torch.randn((B, n, DK + 64), generator=g).to(BF16).to(DEV)
    wide[..., 64:] = kv.to(DEV)
    got = rapid.latent_append(wide[..., 64:], cache, _ints(prefix), inv.to(DEV), q=q, q_out=q_out,
                              kv_weight=None if w is None else w.to(DEV), eps=eps, interleaved=interleaved,
                              row_offset=None if offsets is None else _ints(offsets),
                              n_rows=None if counts is None else _ints(counts))
    torch.cuda.synchronize()
    after = cache.cpu()
    for b in range(B):
        m = n if counts is None else counts[b]
        P = prefix[b]
        fits = 0 <= m <= n and P >= 0 and P + m <= cap
        m = m if fits else 0
        # rows that are not written stay, bit for bit
        rest = torch.ones(cap, dtype=torch.bool)
        rest[max(P, 0):max(P, 0) + m] = False
        assert torch.equal(after[b, rest].view(torch.uint8), before[b, rest].view(torch.uint8)), b
        if H:
            out = got[b].double().cpu()
            if q_kind == "strided":
                assert torch.equal(Q[b, ..., :DC], Q_before[b, ..., :DC])
                assert torch.equal(Q[b, :, m:], Q_before[b, :, m:])
            elif q_kind == "in place":
                assert torch.equal(q[b, m:], q_before[b, m:])
        if m == 0:
            continue
        pos = [P + (i if offsets is None else offsets[b][i]) for i in range(m)]
        # fp32: at most 40 roundings of the size of the values that go in, then one to bf16
        def close(x, ref, size, what):
            arith = 40 * 2.0 ** -24 * size
            err = (x - ref).abs()
            assert (err <= arith + BF16_HALF * (ref.abs() + arith)).all(), (what, b, float(err.max()))
        if H:
            ref, size = _latent.turn(q_before[b, :m].cpu(), pos, inv, interleaved)
            close(out[:m], ref, size, "q")
        ref, size = _latent.turn(kv[b, :m, DC:], pos, inv, interleaved)
        x = _latent.norm(kv[b, :m, :DC], w, eps)
        rows = after[b, P:P + m]
        if not q8:
            close(rows[:, DC:].double(), ref, size, "key")
            close(rows[:, :DC].double(), x, x.abs(), "latent")
            continue
        code, rope, scale = _latent.parts(rows)
        close(rope.double(), ref, size, "key")
        top = x.abs().unflatten(-1, (4, 128)).amax(-1)
        arith = 40 * 2.0 ** -24
        lo, hi = _latent.group_scale(top * (1 - arith)), _latent.group_scale(top * (1 + arith))
        s = scale.double()
        assert ((s == lo) | (s == hi)).all(), b
        wide_s = s.repeat_interleave(128, -1)
        v = code.double() * wide_s
        # half a step of e4m3: 2^-4 of the value, or 2^-10 of the scale
        half = torch.maximum(x.abs() * (1 + arith) * 2.0 ** -4, wide_s * 2.0 ** -10)
        assert ((v - x).abs() <= half + arith * x.abs()).all(), b
        if w is None:             # nothing is computed: the codes are the nearest, ties to even
            assert torch.equal(s, _latent.group_scale(top))
            want = (x / wide_s).float().to(torch.float8_e4m3fn)
            assert torch.equal(want.view(torch.uint8), code.contiguous().view(torch.uint8))


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("B,n,H,interleaved,weight,q_kind", [
    (1, 1, 1, False, True, "strided"), (1, 11, 16, True, True, "strided"), (3, 7, 9, False, False, "in place"),
    (2, 64, 128, False, True, "new"), (2, 130, 0, True, True, "new"), (1, 1000, 3, True, False, "in place")])
def test_append(q8, B, n, H, interleaved, weight, q_kind):
    prefix = [5 + 13 * b for b in range(B)]
    _check_append(q8, B, n, H, prefix, max(prefix) + n + 3, interleaved, weight, q_kind=q_kind)


@pytest.mark.parametrize("q8", [False, True])
def test_append_ragged_tree_and_far_positions(q8):
    n = 12
    offsets = [[i // 2 for i in range(n)], [(1 << 30) + 3 * i for i in range(n)], [-i for i in range(n)]]
    _check_append(q8, 3, n, 8, [0, 100, 40], 112, offsets=offsets, counts=[12, 5, 0], interleaved=True)
    _check_append(q8, 3, n, 8, [0, 100, 40], 112, offsets=offsets, counts=[1, 12, 11])


def test_append_extreme_values():
    g = _gen(4)
    kv = torch.randn((1, 8, DK), generator=g)
    kv[0, 0, :DC] = 0                                   # zeros: scale 1
    kv[0, 1, :DC] *= 1e-30                              # scale 2^-64
    kv[0, 2, :DC] *= 1e30
    kv[0, 3, :128] *= 1e10                              # groups far apart
    kv[0, 4, :DC] = 448.0 * 2 ** -5                     # the largest code, scale a power below
    kv[0, 5, :DC] = 1.0625 * 16                         # ties
    _check_append(True, 1, 8, 1, [3], 16, weight=False, kv=kv.to(BF16))
    _check_append(True, 1, 8, 1, [3], 16, weight=True, kv=kv.to(BF16), eps=0.5)


def test_append_q8_holds_groups_that_are_not_finite_as_nan():
    kv = torch.randn((1, 3, DK), generator=_gen(5)).to(BF16)
    kv[0, 0, 130], kv[0, 1, 511] = NAN, -INF
    cache = torch.zeros((1, 4, 656), dtype=torch.uint8, device=DEV)
    rapid.latent_append(kv.to(DEV), cache, _ints([0]), _inv_freq(None).to(DEV))
    got = rapid.latent_read(cache, None, 3)[0].cpu()
    bad = torch.zeros((3, DK), dtype=torch.bool)
    bad[0, 128:256] = bad[1, 384:512] = True
    assert torch.equal(torch.isnan(got), bad)


@pytest.mark.parametrize("q8", [False, True])
def test_append_leaves_sequences_alone_that_do_not_fit(q8):
    for prefix, counts in (([10, 12, -1], None), ([1, 2, 3], [6, 3, -1])):
        _check_append(q8, 3, 5, 4, prefix, 16, counts=counts)
        torch.cuda.synchronize()
        assert rapid.rapid_device_error(True) == BAD_INPUT


# ---------------------------------------------------------------------------
# Read back, commit
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("n,counts", [(1, None), (4, [4, 0, 3]), (67, [67, 66, 1]), (700, None)])
def test_read(q8, n, counts):
    g = _gen(6)
    first = [3, 0, 20]
    cap = 25 + n
    cache = _latent.make_cache((3, cap), q8, g)
    if q8:       # any code (NaN too) and any finite scale
        code = torch.randint(0, 256, (3, cap, DC), generator=g, dtype=torch.uint8)
        scale = torch.exp(6 * torch.randn((3, cap, 4), generator=g))
        cache = _latent.pack(code.view(torch.float8_e4m3fn), torch.randn((3, cap, DR), generator=g).to(BF16), scale)
        c, r, s = _latent.parts(cache)
        want = torch.cat([(c.float() * s.repeat_interleave(128, -1)).to(BF16), r], -1)
    else:
        want = cache
    out = torch.full((3, n, DK), 7.0, dtype=BF16, device=DEV)
    rapid.latent_read(cache.to(DEV), _ints(first), n, n_rows=None if counts is None else _ints(counts), out=out)
    out = out.cpu()
    for b in range(3):
        m = n if counts is None else counts[b]
        assert torch.equal(out[b, :m].nan_to_num(nan=1e30), want[b, first[b]:first[b] + m].nan_to_num(nan=1e30))
        assert (out[b, m:] == 7.0).all()
    # from the first row
    assert torch.equal(rapid.latent_read(cache.to(DEV), None, 2).cpu().nan_to_num(nan=1e30), want[:, :2].nan_to_num(nan=1e30))


def test_read_leaves_sequences_alone_that_do_not_fit():
    cache = _latent.make_cache((4, 16), False, _gen(7)).to(DEV)
    out = torch.full((4, 5, DK), 7.0, dtype=BF16, device=DEV)
    rapid.latent_read(cache, _ints([12, -1, 3, 11]), 5, n_rows=_ints([5, 5, 6, 5]), out=out)
    assert (out[:3] == 7.0).all() and torch.equal(out[3], cache[3, 11:])
    torch.cuda.synchronize()
    assert rapid.rapid_device_error(True) == BAD_INPUT


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("layers,n_q", [(1, 2), (3, 6), (5, 33), (128, 64)])
def test_commit(q8, layers, n_q):
    g = _gen(layers)
    B, cap = 5, n_q + 9
    caches = torch.stack([_latent.make_cache((B, cap), q8, g) for _ in range(layers)])
    prefix = [9, 0, 4, 1, 7]
    acc = [n_q - 1, 0, n_q // 2, max(1, n_q // 3), min(2, n_q - 1)]
    path = torch.full((B, n_q), -1, dtype=torch.int32)
    for b in range(B):
        path[b, :acc[b]] = (1 + torch.randperm(n_q - 1, generator=g)[:acc[b]]).sort().values
    path[4, :acc[4]] = torch.arange(1, acc[4] + 1)          # a chain: nothing moves
    dev = [c.to(DEV) for c in caches]
    rapid.LatentLayerTable(dev).commit(_ints(prefix), path.to(DEV), _ints(acc))
    want = caches.clone()
    for b in range(B):
        for k in range(acc[b]):
            want[:, b, prefix[b] + 1 + k] = caches[:, b, prefix[b] + int(path[b, k])]
    for x, y in zip(dev, want):
        assert torch.equal(x.cpu().view(torch.uint8), y.view(torch.uint8))


def test_commit_refuses_caches_that_overlap():
    room = torch.zeros((3, 2, 16, DK), dtype=BF16, device=DEV)
    rapid.LatentLayerTable([room[2], room[0], room[1]])
    whole = room.view(-1)
    shifted = whole[8:8 + room[0].numel()].view(2, 16, DK)
    for caches in ([room[0], room[0]], [room[1], room[0], room[1]], [room[1], shifted], [shifted, room[1], room[2]]):
        with pytest.raises(rapid.RapidError):
            rapid.LatentLayerTable(caches)


def test_commit_leaves_invalid_sequences_alone():
    caches = _latent.make_cache((6, 16), False, _gen(9))
    dev = caches.to(DEV)
    prefix, acc = [0, 11, -1, 2, 2, 2], [6, 2, 2, 2, 2, 2]
    path = _ints([[2, 3, 4, 5, -1, -1]] * 3 + [[3, 2, -1, -1, -1, -1], [1, 6, -1, -1, -1, -1], [2, 4, -1, -1, -1, -1]])
    rapid.rapid_latent_commit(rapid.LatentLayerTable([dev]), _ints(prefix), path, _ints(acc))
    want = caches.clone()
    want[5, 3], want[5, 4] = caches[5, 4], caches[5, 6]
    assert torch.equal(dev.cpu(), want)
    torch.cuda.synchronize()
    assert rapid.rapid_device_error(True) == BAD_INPUT


# ---------------------------------------------------------------------------
# Absorbed attention
# ---------------------------------------------------------------------------

def _check_attn(Q, cache, prefix, mask=None, scale=_latent.SCALE, **kw):
    O, L = rapid.latent_attn(Q, cache, _ints(prefix), mask, 0.0 if scale == _latent.SCALE else scale, **kw)
    Oe, Le, eO, eL = _latent.attn(Q, cache, prefix, mask, scale)
    err, lerr = (O.double() - Oe).abs(), (L.double() - Le).abs()
    empty = Le == -math.inf
    assert torch.equal(L == -math.inf, empty) and (O[empty] == 0).all()
    assert (err <= eO)[~empty].all(), float((err / eO.clamp(min=1e-30)).max())
    assert (lerr <= eL)[~empty].all(), float((lerr / eL)[~empty].max())
    return O, L


def _inputs(B, H, n, prefix, q8, seed, extra=5, spread=0.5):
    g = _gen(seed)
    Q = torch.randn((B, H, n, DK), generator=g).to(BF16).to(DEV)
    cache = _latent.make_cache((B, max(prefix) + n + extra), q8, g, spread).to(DEV)
    return Q, cache


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("B,H,n,prefix", [
    (1, 1, 1, [0]), (1, 16, 1, [62]), (1, 16, 1, [63]), (1, 16, 1, [64]), (1, 5, 3, [61]), (1, 17, 1, [130]),
    (2, 16, 2, [0, 129]), (3, 5, 7, [1, 64, 500]), (1, 64, 3, [1000]), (2, 128, 11, [300, 77]),
    (1, 3, 64, [127]), (1, 2, 64, [0]), (1, 16, 1, [12345]), (1, 40, 2, [3000]), (6, 16, 1, [3, 900, 0, 63, 64, 4000])])
def test_attn_chain(q8, B, H, n, prefix):
    _check_attn(*_inputs(B, H, n, prefix, q8, seed=B + H + n), prefix)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("B", [33, 77, 200, 700])
def test_attn_many_sequences(q8, B):
    # more than a warp's lanes; more splits than, and as many as, sequences; one split each
    prefix = [(37 * b) % 401 for b in range(B)]
    _check_attn(*_inputs(B, 2, 3, prefix, q8, seed=B), prefix)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("n,prefix", [(1, [0, 5]), (6, [0, 62]), (32, [40, 0]), (64, [0, 100]), (33, [31, 95])])
def test_attn_masks(q8, n, prefix):
    Q, cache = _inputs(2, 20, n, prefix, q8, seed=n)
    g = _gen(n)
    mask = (torch.rand((2, n, n), generator=g) < 0.4).to(torch.uint8)
    mask[0, n // 2] = 0                                  # a row that sees nothing of the step
    mask[1, 0] = 1
    mask[mask != 0] = 255                                # any value that is not zero
    _check_attn(Q, cache, prefix, mask.to(DEV))
    _check_attn(Q, cache, prefix, (mask != 0).to(DEV))   # torch.bool
    _check_attn(Q, cache, prefix, torch.zeros_like(mask).to(DEV))


@pytest.mark.parametrize("q8", [False, True])
def test_attn_scores_that_keep_rising(q8):
    # a scale at which the maximum moves by far more than 2^16 from tile to tile, some rows later
    prefix = [700]
    Q, cache = _inputs(1, 24, 5, prefix, q8, seed=3)
    Q[0, ::3] *= 0.01
    for scale in (0.3, 2.0):
        _check_attn(Q, cache, prefix, scale=scale)


def test_attn_q8_scales_of_any_size():
    g = _gen(8)
    n, P = 3, 200
    cache = _latent.make_cache((1, P + n), True, g)
    code, rope, scale = _latent.parts(cache)
    scale = scale * torch.exp2(torch.randint(-40, 3, scale.shape, generator=g).float())
    scale[0, 5], scale[0, 70, 1], scale[0, 130, 2] = 2.0 ** -64, 2.0 ** 9, 2.0 ** 30   # past 2^7: two steps
    code = code.clone()
    code.view(torch.uint8)[0, 9] = torch.arange(512, dtype=torch.int32).to(torch.uint8) & 0x87   # subnormal codes
    cache = _latent.pack(code, rope, scale)
    Q = torch.randn((1, 16, n, DK), generator=g)
    Q[..., 128:384] *= 2.0 ** -12                          # keeps the large groups' scores in range
    Q[..., 256:384] *= 2.0 ** -22
    _check_attn(Q.to(BF16).to(DEV), cache.to(DEV), [P])


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("n,prefix", [(5, [0, 59, 64]), (64, [0, 33, 70])])
def test_attn_hidden_rows_and_other_queries_may_hold_anything(q8, n, prefix):
    Q, cache = _inputs(3, 16, n, prefix, q8, seed=n, extra=70)
    g = _gen(11)
    mask = (torch.rand((3, n, n), generator=g) < 0.5).to(torch.uint8).to(DEV)
    mask[:, :, 2] = 0                                     # a row of the step that nobody sees
    mask[:, :, 3] = 0
    mask[:, 1, 3] = 1                                     # one that one query sees
    clean_O, clean_L = _check_attn(Q, cache, prefix, mask)
    x = cache.clone()
    for b, P in enumerate(prefix):
        for row, v in ((P + 2, NAN), (P + 3, NAN)):
            if q8:
                _latent.parts(x)[2][b, row] = v
                _latent.parts(x)[1][b, row] = INF
            else:
                x[b, row] = v
                x[b, row, ::2] = INF
        x[b, P + n:] = 0xff if q8 else NAN                # behind the step
    Q2 = Q.clone()
    Q2[:, 3] = NAN                                        # another head's queries
    Q2[:, 4, 0] = INF
    O, L = rapid.latent_attn(Q2, x, _ints(prefix), mask)
    hit = torch.zeros_like(clean_L, dtype=torch.bool)
    hit[:, :, 1] = True
    hit[:, 3] = True
    hit[:, 4, 0] = True
    assert torch.isnan(L[:, 3][clean_L[:, 3] > -INF]).all() and torch.isnan(O[:, :3, 1]).all() and torch.isnan(L[:, :3, 1]).all()
    assert torch.equal(O[~hit], clean_O[~hit]) and torch.equal(L[~hit], clean_L[~hit])


@pytest.mark.parametrize("q8", [False, True])
def test_attn_a_bad_history_row_reaches_every_query(q8):
    prefix = [300]
    Q, cache = _inputs(1, 16, 2, prefix, q8, seed=5)
    if q8:
        _latent.parts(cache)[2][0, 100, 3] = NAN
    else:
        cache[0, 100, 500] = NAN
    O, L = rapid.latent_attn(Q, cache, _ints(prefix))
    assert torch.isnan(O).all() and torch.isnan(L).all()


def test_attn_lengths_out_of_range_are_clamped():
    Q, cache = _inputs(3, 4, 3, [100, 100, 100], False, seed=6, extra=0)
    O, L = rapid.latent_attn(Q, cache, _ints([-5, 1 << 30, 50]))
    want = rapid.latent_attn(Q, cache, _ints([0, 100, 50]))
    torch.cuda.synchronize()
    assert rapid.rapid_device_error(True) == BAD_INPUT
    assert torch.equal(O, want[0]) and torch.equal(L, want[1])


def test_attn_offsets_past_32_bits():
    # the last rows of a cache of 4.7 GB, behind a history that is mostly not read
    n, cap = 2, 1 << 21
    cache = torch.empty((2, cap, DK), dtype=BF16, device=DEV)
    g = _gen(12)
    part = _latent.make_cache((1, 300), False, g).to(DEV)
    cache[1, -300:] = part[0]
    cache[1, :300] = part[0]
    Q = torch.randn((1, 16, n, DK), generator=g).to(BF16).to(DEV).expand(2, -1, -1, -1).contiguous()
    out = torch.empty((2, 5, DK), dtype=BF16, device=DEV)
    rapid.latent_read(cache, _ints([0, cap - 5]), 5, out=out)
    assert torch.equal(out[1], part[0, -5:])
    O, L = rapid.latent_attn(Q, cache, _ints([0, 250]))
    want, _, eO, _ = _latent.attn(Q[1:], part, [250])
    assert ((O[1:].double() - want).abs() <= eO).all()


def test_attn_is_the_same_twice_and_leaves_its_inputs_alone():
    prefix = [900, 17]
    Q, cache = _inputs(2, 32, 4, prefix, True, seed=7)
    keep = Q.clone(), cache.clone()
    a = rapid.latent_attn(Q, cache, _ints(prefix))
    out, lse = torch.empty_like(a[0]), torch.empty_like(a[1])
    ws = torch.full((rapid.rapid_latent_attn_workspace_size(2, 32, 4, cache.shape[1], rapid.RAPID_CACHE_LATENT_Q8),),
                    255, dtype=torch.uint8, device=DEV)
    b = rapid.latent_attn(Q, cache, _ints(prefix), out=out, lse=lse, workspace=ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert torch.equal(Q, keep[0]) and torch.equal(cache, keep[1])
    with pytest.raises(rapid.RapidError):
        rapid.latent_attn(Q, cache, _ints(prefix), workspace=ws[:-1])
    with pytest.raises(rapid.RapidError):
        rapid.latent_attn(Q, cache[:1], _ints(prefix))
    with pytest.raises(rapid.RapidError):
        rapid.latent_attn(Q[..., :512], cache, _ints(prefix))
