"""Plain 64-bit forms of the latent cache's operators, for the tests, written from the definitions
(rapid.h): no code shared with the library.  Those of the attention calls come with the error that
the kernels' arithmetic may add, counted from the roundings they make.
"""
import math

import torch

DC, DR, DK, HEAD, GROUP = 512, 64, 576, 128, 128
Q8_ROW = 656
BF16_HALF = 2.0 ** -8       # half a step, relative, at most
SCALE = 192 ** -0.5
# A tensor-core sum adds 16 products to an fp32 accumulator at a time; each such step may lose
# 2^-23 (truncation) of the sum of magnitudes so far, and as much inside.
STEP = 2.0 ** -22


def parts(cache):
    """Codes, rotated values and scales of 8-bit rows."""
    return (cache[..., :DC].view(torch.float8_e4m3fn), cache[..., DC:DC + 2 * DR].view(torch.bfloat16),
            cache[..., DC + 2 * DR:].view(torch.float32))


def values(cache):
    """Rows in 64 bits."""
    if cache.dtype != torch.uint8:
        return cache.double()
    code, rope, scale = parts(cache)
    return torch.cat([code.double() * scale.double().repeat_interleave(GROUP, -1), rope.double()], -1)


def pack(code, rope, scale):
    """8-bit rows of their parts (e4m3, bf16, float32)."""
    return torch.cat([code.contiguous().view(torch.uint8), rope.contiguous().view(torch.uint8),
                      scale.contiguous().view(torch.uint8)], -1)


def group_scale(top):
    """2^ceil(log2(top / 448)), an exponent below -64 as -64, 1 for zero; float64 in and out."""
    m, e = torch.frexp(top / 448)                     # top / 448 = m 2^e, 1/2 <= m < 1
    e = torch.where(m == 0.5, e - 1, e).clamp(min=-64)
    return torch.where(top > 0, torch.ldexp(torch.ones_like(top), e), torch.ones_like(top))


def make_cache(shape, q8, g, spread=0.5):
    """Random rows on the CPU, as a norm leaves them."""
    x = torch.randn((*shape, DK), generator=g)
    x *= torch.exp(spread * torch.randn((DK,), generator=g))
    if not q8:
        return x.bfloat16()
    y = x[..., :DC].unflatten(-1, (4, GROUP))
    s = group_scale(y.abs().amax(-1).double()).float()
    return pack((y / s[..., None]).flatten(-2).to(torch.float8_e4m3fn), x[..., DC:].bfloat16(), s)


def chain(B, n):
    return torch.ones((n, n), dtype=torch.uint8).tril().expand(B, n, n).contiguous()


def _softmax(x):
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total > 0, total, torch.ones_like(total)), (total.log() + top)[..., 0]


def _bounds(x, mag, p, v, o, lse, keys, depth):
    """Errors of O and LSE.  x: scaled scores (-inf: hidden), mag: scale * sum |q k|, p: probabilities,
    v: values; depth: 16-wide steps of a score's sum.

    A score is off by depth steps of its magnitudes; its exponential also by the argument's
    rounding (2^-24 of the distance to the reference, in units where that is at most the spread of
    the scores; twice, for the two factors of the log2 domain) and the exponential's 2^-22.  P is
    rounded to bf16 once; the sum over keys takes a step for 16 of them, the sum of
    probabilities at most one fp32 rounding for each 8 (a lane's share of a tile) and tile; parts
    are joined by some 2^-20; O is rounded to bf16."""
    seen = x > -math.inf
    spread = torch.where(seen, (x - x.masked_fill(~seen, math.inf).amin(-1, keepdim=True)).abs(),
                         torch.zeros_like(x)).amax(-1)
    # a reference may stay 16 ln 2 below the row's maximum
    d = torch.where(seen, mag, torch.zeros_like(mag)).amax(-1) * depth * STEP + (spread + 12) * 2.0 ** -23 + 2.0 ** -21
    total = keys / 8 * 2.0 ** -24 + 2.0 ** -20
    big = p @ v.abs()
    eo = big * (BF16_HALF + 2 * d[..., None] + keys / 16 * STEP + total)
    return eo + BF16_HALF * (o.abs() + eo), d + total + lse.abs().nan_to_num(0, 0, 0) * 2.0 ** -21


def attn(Q, cache, prefix_len, mask=None, scale=SCALE):
    """(O, LSE, bound of O's error, bound of LSE's) of the absorbed form, in float64."""
    B, H, n, _ = Q.shape
    O = torch.zeros((B, H, n, DC), dtype=torch.float64, device=Q.device)
    L = torch.full((B, H, n), -math.inf, dtype=torch.float64, device=Q.device)
    eO, eL = torch.zeros_like(O), torch.zeros_like(L)
    for b in range(B):
        P = int(prefix_len[b])
        rows = values(cache[b, :P + n])
        seen = torch.ones((n, P + n), dtype=torch.bool, device=Q.device)
        seen[:, P:] = torch.ones((n, n), device=Q.device).tril().bool() if mask is None else mask[b] != 0
        for h in range(H):
            q = Q[b, h].double()
            # hidden rows may hold anything
            x = (q @ rows.T * scale).masked_fill(~seen, -math.inf)
            p, lse = _softmax(x)
            clean = rows[:, :DC].clone()
            clean[~seen.any(0)] = 0
            o = torch.stack([p[i] @ torch.where(seen[i][:, None], rows[:, :DC], torch.zeros_like(clean))
                             for i in range(n)]) if not torch.isfinite(rows).all() else p @ clean
            O[b, h], L[b, h] = o, lse
            eO[b, h], eL[b, h] = _bounds(x, q.abs() @ rows.abs().T * scale, p, clean, o, lse, P + n, DK // 16 + 1)
    return O, L, eO, eL


def prefill(Q, K, V, K_rope, prefix_len, n_rows=None, scale=SCALE):
    """(O, LSE, bounds) of the expanded form; rows behind n_rows are zero."""
    B, n, H, _ = Q.shape
    O = torch.zeros((B, n, H, HEAD), dtype=torch.float64, device=Q.device)
    L = torch.zeros((B, H, n), dtype=torch.float64, device=Q.device)
    eO, eL = torch.zeros_like(O), torch.zeros_like(L)
    for b in range(B):
        P, m = int(prefix_len[b]), n if n_rows is None else int(n_rows[b])
        seen = torch.ones((m, P + m), dtype=torch.bool, device=Q.device).tril(P)
        for h in range(H):
            k = torch.cat([K[b, :P + m, h], K_rope[b, :P + m]], -1).double()
            v, q = V[b, :P + m, h].double(), Q[b, :m, h].double()
            x = (q @ k.T * scale).masked_fill(~seen, -math.inf)
            p, lse = _softmax(x)
            o = torch.stack([p[i] @ torch.where(seen[i][:, None], v, torch.zeros_like(v)) for i in range(m)]
                            ) if not torch.isfinite(v).all() else p @ v
            O[b, :m, h], L[b, h, :m] = o, lse
            eO[b, :m, h], eL[b, h, :m] = _bounds(x, q.abs() @ k.abs().T * scale, p, v, o, lse, P + m, 192 // 16 + 1)
    return O, L, eO, eL


def turn(x, pos, inv_freq, interleaved):
    """Rows x [n, ..., 64] rotated by positions [n] in float64, and |a| + |b| of each pair."""
    x = x.double()
    # whole turns leave the angle alone: in integers, in units of 2^-60 turns
    ang = torch.tensor([[float((int(p) * round(float(f) / (2 * math.pi) * 2 ** 60)) % 2 ** 60) * 2.0 ** -60
                         * 2 * math.pi for f in inv_freq] for p in pos], dtype=torch.float64, device=x.device)
    shape = (len(pos),) + (1,) * (x.dim() - 2) + (DR // 2,)
    c, s = ang.cos().view(shape), ang.sin().view(shape)
    ia = torch.arange(0, DR, 2) if interleaved else torch.arange(DR // 2)
    ib = ia + 1 if interleaved else ia + DR // 2
    y, size = torch.empty_like(x), torch.empty_like(x)
    y[..., ia], y[..., ib] = x[..., ia] * c - x[..., ib] * s, x[..., ib] * c + x[..., ia] * s
    size[..., ia] = size[..., ib] = x[..., ia].abs() + x[..., ib].abs()
    return y, size


def norm(x, weight, eps):
    x = x.double()
    return x if weight is None else x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()
