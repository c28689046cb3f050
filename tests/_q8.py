"""Plain 64-bit forms of the 8-bit cache's operators, on the CPU, for the tests.

Written from the definitions (rapid.h): loops over sequences and heads, no code shared with
the library.  Each comes with the error that the kernels' arithmetic may add, counted from
the roundings they make.
"""
import math

import numpy as np
import torch

PAGE = 64
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # relative, at most


def append(q, k, v, K, V, Q, prefix_len, inv_freq=None, q_weight=None, k_weight=None, eps=1e-6,
           interleaved=False, pos_offset=None, row_offset=None, n_rows=None):
    """(Q, K, V) after the call in float64, and the bounds of Q's and K's errors.

    fp32 arithmetic: the sum of squares, its square root and the two products of the norm
    are at most 24 roundings, the sine and cosine 4, the rotation 3, each 2^-24 relative to
    |a| + |b| of the rotated pair; then half a step of the output type."""
    dt = q.dtype
    B, n, Hq, d = q.shape
    Q, K, V = (t.double().clone() for t in (Q, K, V))
    eQ, eK = torch.zeros_like(Q), torch.zeros_like(K)
    rot = 0 if inv_freq is None else 2 * len(inv_freq)
    for b in range(B):
        m = n if n_rows is None else int(n_rows[b])
        p0 = int(prefix_len[b])
        if not 0 <= m <= n or p0 < 0 or p0 + m > K.shape[2]:
            continue
        for i in range(m):
            pos = p0 + (i if row_offset is None else int(row_offset[b, i]))
            pos += 0 if pos_offset is None else int(pos_offset[b])
            for x, w, out, err, row in ((q, q_weight, Q, eQ, i), (k, k_weight, K, eK, p0 + i)):
                y = x[b, i].double()
                if w is not None:
                    y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double()
                size = y.abs()
                if rot:
                    # the angle modulo a turn in extended precision: exact enough at any position
                    turns = [math.fmod(pos * float(f), 2 * math.pi) if abs(pos) < 1 << 20 else
                             float(np.fmod(np.longdouble(pos) * np.longdouble(float(f)),
                                           2 * np.longdouble("3.14159265358979323846264338327950288")))
                             for f in inv_freq]
                    c = torch.tensor([math.cos(t) for t in turns], dtype=torch.float64)
                    s = torch.tensor([math.sin(t) for t in turns], dtype=torch.float64)
                    ia = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
                    ib = ia + 1 if interleaved else ia + rot // 2
                    a, e = y[:, ia].clone(), y[:, ib].clone()
                    y[:, ia], y[:, ib] = a * c - e * s, e * c + a * s
                    both = size[:, ia] + size[:, ib]
                    size[:, ia], size[:, ib] = both, both
                out[b, :, row] = y
                # without norm and rotation a row is copied
                arith = 32 * 2.0 ** -24 * size if (rot or w is not None) else 0 * size
                err[b, :, row] = arith + HALF_STEP[dt] * (y.abs() + arith)
            V[b, :, p0 + i] = v[b, i].double()
    return Q, K, V, eQ, eK


def e4m3_round(x):
    """Nearest e4m3 value of |x| <= 448 (ties to the even code), and NaN for NaN."""
    x = np.asarray(x, np.float64)
    a = np.abs(x)
    _, e = np.frexp(np.maximum(a, 2.0 ** -6))       # a = m 2^e, m in [1/2, 1)
    step = 2.0 ** (e - 4.0)                         # 8 values per power of two
    return np.where(np.isnan(x), np.nan, np.round(x / step) * step)


def block_scale(top):
    """Smallest power of two s with top <= 448 s, at least 2^-64; 1 for zero."""
    if top == 0:
        return 1.0
    e = -64
    while 448.0 * 2.0 ** e < top:
        e += 1
    return 2.0 ** e


def seal(K, V, pages, scales, page_table, sealed_len, tail_len, keep):
    """One layer, in place on float64 numpy arrays (pages hold values, not codes); new
    (sealed_len, tail_len) and whether an input was refused."""
    B, Hkv, cap, d = K.shape
    sealed2, tail2, bad = sealed_len.copy(), tail_len.copy(), False
    for b in range(B):
        S, P = int(sealed_len[b]), int(tail_len[b])
        if P < 0 or P > cap or S < 0 or S % PAGE:
            bad = True
            continue
        n_b = max(0, P - keep) // PAGE
        ids = page_table[b, S // PAGE:S // PAGE + n_b]
        if len(ids) < n_b or (ids < 0).any() or (ids >= pages.shape[0]).any():
            bad = True
            continue
        for j in range(n_b):
            for g in range(Hkv):
                for side, t in enumerate((K, V)):
                    x = t[b, g, j * PAGE:(j + 1) * PAGE].copy()
                    x[~np.isfinite(x)] = np.nan
                    top = np.nanmax(np.abs(x)) if np.isfinite(x).any() else 0.0
                    s = block_scale(top)
                    scales[ids[j], g, side] = s
                    pages[ids[j], g, side] = e4m3_round(x / s)
        if n_b:
            rest = P - n_b * PAGE
            for t in (K, V):
                t[b, :, :rest] = t[b, :, n_b * PAGE:P].copy()
        sealed2[b], tail2[b] = S + n_b * PAGE, P - n_b * PAGE
    return sealed2, tail2, bad


def attn(Q, K, V, pages, scales, page_table, sealed_len, tail_len, mask=None, softmax_scale=None):
    """O, LSE in float64 and the bounds of their errors.

    Scores: d products, exact in fp32, summed in fp32 (2^-23 per addition, the tensor core's
    truncation included) and scaled twice: ds.  exp2 is good to 2^-21 relative.  The sums
    over keys: 2^-24 per addition and key.  Probabilities are rounded to fp16 over pages
    (2^-11, and 2^-31 of the largest where fp16 runs out of exponents) and to bf16 over
    tail rows (2^-8) in the bf16 kernel, not at all in the fp32 one."""
    dt = Q.dtype
    B, Hq, n, d = Q.shape
    Hkv = K.shape[1]
    G = Hq // Hkv
    c = 1 / math.sqrt(d) if softmax_scale is None else softmax_scale
    O = torch.zeros(Q.shape, dtype=torch.float64)
    L = torch.zeros(Q.shape[:3], dtype=torch.float64)
    eO, eL = torch.zeros_like(O), torch.zeros_like(L)
    p_page, p_tail = (2.0 ** -11, 2.0 ** -8) if dt == torch.bfloat16 else (0.0, 0.0)
    for b in range(B):
        ids = page_table[b, :int(sealed_len[b]) // PAGE].long()
        t = int(tail_len[b])
        S = len(ids) * PAGE
        seen = torch.ones((n, S + t + n), dtype=torch.bool)
        seen[:, S + t:] = torch.ones((n, n)).tril().bool() if mask is None else mask[b].bool()
        for g in range(Hkv):
            kv = pages.view(torch.uint8)[ids, g].view(pages.dtype).double() * scales[ids, g].double()[..., None, None]
            keys = torch.cat([kv[:, 0].reshape(-1, d), K[b, g, :t + n].double()])
            vals = torch.cat([kv[:, 1].reshape(-1, d), V[b, g, :t + n].double()])
            for h in range(g * G, (g + 1) * G):
                for i in range(n):
                    on = seen[i]
                    if not on.any():
                        L[b, h, i] = -math.inf
                        continue
                    q, k, v = Q[b, h, i].double(), keys[on], vals[on]
                    x = (k @ q) * c
                    lse = torch.logsumexp(x, 0)
                    p = torch.exp(x - lse)
                    O[b, h, i], L[b, h, i] = p @ v, lse
                    N = len(x)
                    ds = c * float((k.abs() @ q.abs()).max()) * (d + 4) * 2.0 ** -23
                    ds += float(x.abs().max()) * 2.0 ** -22 + 2.0 ** -21
                    A = p @ v.abs()
                    page = on.nonzero()[:, 0] < S
                    rp = p_page * (p[page] @ v[page].abs()) + p_tail * (p[~page] @ v[~page].abs())
                    e = A * (2 * ds + N * 2.0 ** -24 + 2.0 ** -20) + rp
                    if p_page:
                        e = e + N * 2.0 ** -31 * torch.nan_to_num(v, 0.0, 0.0, 0.0).abs().max()
                    eO[b, h, i] = e + HALF_STEP[dt] * (O[b, h, i].abs() + e)
                    eL[b, h, i] = ds + N * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -22 * abs(float(lse))
    return O, L, eO, eL


def check(got, ref, err, what):
    got, ref = got.detach().cpu().double(), ref
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN in other places"
    fin = torch.isfinite(ref)
    same = got[~fin & ~torch.isnan(ref)] == ref[~fin & ~torch.isnan(ref)]
    assert bool(same.all()), f"{what}: infinities differ"
    over = ((got - ref).abs() - err)[fin]
    assert over.numel() == 0 or float(over.max()) <= 0, (
        f"{what}: {float((got - ref).abs()[fin].max())} off, over the bound by {float(over.max())}")


def cache(B, Hkv, d, dtype, blocks, tails, n, seed, spare=2, n_pages=None, scale_spread=0):
    """A random cache on the CPU: dict of K, V (tails), pages, scales, page_table, lengths."""
    g = torch.Generator().manual_seed(seed)
    per = max(1, max(blocks) + spare)
    n_pages = B * per + 1 if n_pages is None else n_pages
    cap = (max(tails) + n + 15) // 16 * 16
    raw = torch.randn((n_pages, Hkv, 2, PAGE, d), generator=g)
    e = torch.randint(-8 - scale_spread, -6 + scale_spread + 1, (n_pages, Hkv, 2), generator=g)
    scales = torch.pow(2.0, e.float())
    codes = (raw * (2.0 ** 7)).clamp(-448, 448).to(torch.float8_e4m3fn)
    table = torch.randperm(n_pages, generator=g)[:B * per].to(torch.int32).view(B, per)
    return dict(K=torch.randn((B, Hkv, cap, d), generator=g).to(dtype),
                V=torch.randn((B, Hkv, cap, d), generator=g).to(dtype), pages=codes, scales=scales,
                page_table=table.contiguous(),
                sealed_len=torch.tensor([PAGE * x for x in blocks], dtype=torch.int32),
                tail_len=torch.tensor(tails, dtype=torch.int32))
