"""Cases of the operators around a latent key/value cache, with their plain forms.

A target with a latent cache keeps one row a token for all its heads: 512 values of a normed
latent vector, from which keys and values of every head follow by matrix products, and 64
values of a rotated key that all heads share.  A row is held as 576 bf16 values, or in 656
bytes: 512 e4m3 codes, the 64 rotated values in bf16, and four fp32 powers of two, one for
each 128 codes.

* ``append``  a step's or a chunk's projection rows: norm and rotation, quantised as they are
              written to the cache; the rotated part of the queries (``rapid.latent_append``);
* ``attn``    the absorbed form: verify attention on the rows themselves, keys of 576 and
              values of 512 (``rapid.latent_attn``);
* ``commit``  the accepted path's rows of every layer move next to the root
              (``rapid.LatentLayerTable.commit``);
* ``read``    rows of the cache back in bf16 (``rapid.latent_read``);
* ``prefill`` the expanded form: causal attention of a prompt chunk, keys of 128 for each head
              and 64 shared, values of 128 (``rapid.latent_prefill_attn``).

``run`` takes a state from ``prepare`` through one of them: with ``own`` false as elementary
torch operations in 32 bits, with ``own`` true as the library's calls.  ``exact`` gives the
same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

DC, DR = 512, 64             # latent and rotated values of a row
DK = DC + DR
NOPE, DV = 128, 128          # per-head key and value width of the expanded form
GROUP = 128                  # codes that share a scale
ROW_BYTES = DC + 2 * DR + 4 * (DC // GROUP)
E4M3_MAX = 448.0
SCALE_EXP_MIN = -64
THETA = 500000.0
EPS = 1e-6
SCALE = (NOPE + DR) ** -0.5


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _append(name, B, n, H, q8, base, interleaved=False, tree=False, ragged=False):
    return dict(name=name, op="append", B=B, n=n, H=H, q8=q8, base=base, interleaved=interleaved,
                tree=tree, ragged=ragged)


def _attn(name, B, n, H, q8, lo, hi, tree=False):
    return dict(name=name, op="attn", B=B, n=n, H=H, q8=q8, lo=lo, hi=hi, tree=tree)


def _commit(name, layers, B, n, q8, base):
    return dict(name=name, op="commit", layers=layers, B=B, n=n, q8=q8, base=base)


def _read(name, B, n, q8, base, ragged=False):
    return dict(name=name, op="read", B=B, n=n, q8=q8, base=base, ragged=ragged)


def _prefill(name, B, n, H, lo, hi, ragged=False):
    return dict(name=name, op="prefill", B=B, n=n, H=H, lo=lo, hi=hi, ragged=ragged)


def listed():
    return [
        # one verify step of an 11-node chain of a 128-head target at 120K, 8-bit rows: a call
        # of a few microseconds between two matrix products
        _append("append_step_q8_128h", 1, 11, 128, True, 122880),
        # prefill chunks of different lengths, interleaved pairs: bandwidth counts
        _append("append_ragged_bf16_32h", 3, 4095, 32, False, 1021, interleaved=True, ragged=True),
        # one token of a 16-head target over a short history: latency
        _attn("attn_decode_1k_16h", 1, 1, 16, False, 1021, 1021),
        # one token of a 128-head target at 120K, 8-bit rows
        _attn("attn_decode_120k_128h_q8", 1, 1, 128, True, 122880, 122880),
        # the 11-node chain of the same target on bf16 rows: 1408 query rows
        _attn("attn_chain_120k_128h", 1, 11, 128, False, 122869, 122869),
        # a tree of 32 nodes of a 16-head target on four ragged histories of 32K to 96K
        _attn("attn_tree_ragged_16h_q8", 4, 32, 16, True, 32768, 98303, tree=True),
        # the accepted paths of four 32-node trees, 32 layers
        _commit("commit_tree_32layers_q8", 32, 4, 32, True, 4099),
        # sixteen sequences with 64-node trees, 60 layers of bf16 rows
        _commit("commit_batch_60layers", 60, 16, 64, False, 513),
        # the start of three cached prompts, for the products of the expanded form
        _read("read_ragged_3x1999", 3, 1999, False, 77, ragged=True),
        # a whole 120K history in 8 bits
        _read("read_history_120k_q8", 1, 122880, True, 0),
        # the last chunks of three prompts behind histories of up to 12K
        _prefill("prefill_ragged_16h", 3, 999, 16, 0, 12001, ragged=True),
        # a prompt of 8K from its start, 32 heads
        _prefill("prefill_8k_32h", 1, 8192, 32, 0, 0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "attn", "commit", "read", "prefill", "prefill"])
    q8 = rng.random() < 0.5
    B = rng.randint(1, 6)
    H = rng.choice([8, 16, 20, 32, 64, 128])
    if op == "append":
        tree = rng.random() < 0.4
        # 8-bit rows: up to 1024 a call (a scale that rests on a rounding would differ by two)
        n = rng.randint(1, 64) if tree else _log_int(rng, 1, (1024 if q8 else 12288) // B)
        c = _append("", B, n, H, q8, _log_int(rng, 1, 65536), rng.random() < 0.4, tree,
                    rng.random() < 0.4)
    elif op == "attn":
        n = rng.choice([1, rng.randint(2, 16), rng.randint(2, 16), rng.randint(17, 64)])
        most = min(122880 // B, 122880 * 1408 // (H * n * B))
        hi = _log_int(rng, 1, most)
        lo = hi if rng.random() < 0.4 else rng.randint(0, hi)
        c = _attn("", B, n, H, q8, lo, hi, rng.random() < 0.5)
    elif op == "commit":
        n = rng.randint(2, 64)
        c = _commit("", _log_int(rng, 1, 64), rng.randint(1, 16), n, q8, _log_int(rng, 1, 1024))
    elif op == "read":
        c = _read("", B, _log_int(rng, 1, 122880 // B), q8, rng.randint(0, 1000),
                  rng.random() < 0.4)
    else:
        n = _log_int(rng, 1, 4096 // B)
        most = 8192 * 8192 * 32 // (2 * n * H * B) - n
        hi = rng.randint(0, max(0, min(16384, most)))
        lo = hi if rng.random() < 0.4 else rng.randint(0, hi)
        c = _prefill("", B, n, H, lo, hi, rng.random() < 0.4)
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# Lengths of a case's sequences (the case alone decides them)
# ---------------------------------------------------------------------------

def _history(c):
    """History rows of each sequence."""
    B = c["B"]
    if c["op"] in ("append", "commit", "read"):
        return [c["base"] + 37 * b for b in range(B)]
    lo, hi = c["lo"], c["hi"]
    return [hi] if B == 1 else [lo + (hi - lo) * b // (B - 1) for b in range(B)]


def _counts(c):
    """New rows (append, prefill) or rows read of each sequence."""
    n, B = c["n"], c["B"]
    return [n if not c.get("ragged") else max(1, n - n * b // (B + 1)) for b in range(B)]


def _accepted(c):
    """Accepted drafts of each sequence: none, some, as far as a path of odd nodes goes."""
    most = c["n"] // 2
    return [most * (b + 1) // c["B"] for b in range(c["B"])]


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _tree_parents(n, g):
    """Parents and depths of a random tree of depth up to 6 below the root."""
    parent, depth = [-1], [0]
    for i in range(1, n):
        free = [j for j in range(i) if depth[j] < 6]
        j = free[int(torch.randint(len(free), (1,), generator=g))]
        parent.append(j)
        depth.append(depth[j] + 1)
    return parent, depth


def _group_scale(amax):
    """The power of two that brings amax into e4m3's range (1 for a group of zeros)."""
    m, e = torch.frexp(amax)
    e = e - 9 + (m > 0.875).to(e.dtype)   # 448 = 0.875 * 2^9
    e = torch.where(amax > 0, e.clamp(min=SCALE_EXP_MIN), torch.zeros_like(e))
    return torch.ldexp(torch.ones_like(amax), e)


def _pack(latent, rope):
    """8-bit rows of fp32 latents [..., 512] and rope keys [..., 64]."""
    x = latent.unflatten(-1, (DC // GROUP, GROUP))
    scale = _group_scale(x.abs().amax(-1))
    code = (x / scale[..., None]).flatten(-2).to(torch.float8_e4m3fn)
    return torch.cat([code.view(torch.uint8), rope.bfloat16().view(torch.uint8),
                      scale.contiguous().view(torch.uint8)], -1)


def _rows(shape, g, dev):
    """fp32 rows as a norm leaves them: a spread of sizes over the channels."""
    x = torch.randn(shape, generator=g, device=dev)
    x *= torch.exp(0.5 * torch.randn(shape[-1:], generator=g, device=dev))
    return x


def _cache(shape, q8, g, dev):
    x = _rows((*shape, DK), g, dev)
    return _pack(x[..., :DC], x[..., DC:]) if q8 else x.bfloat16()


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    gc = torch.Generator().manual_seed(seed)
    c, s = case, {"case": case}
    B, n = c["B"], c["n"]

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    if c["op"] == "append":
        H = c["H"]
        # one projection gives a query head's 128 plain values and the 64 to rotate, another
        # the latent vector and the shared key
        q = _rows((B, n, H, NOPE + DR), g, dev).bfloat16()
        s["q"] = q[..., NOPE:]
        s["kv"] = _rows((B, n, DK), g, dev).bfloat16()
        s["Q"] = torch.randn((B, H, n, DK), generator=g, device=dev).bfloat16()
        s["q_out"] = s["Q"][..., DC:].transpose(1, 2)
        s["weight"] = (1 + 0.2 * torch.randn(DC, generator=g, device=dev)).bfloat16()
        s["inv_freq"] = (THETA ** (-torch.arange(0, DR, 2, device=dev).double() / DR)).float()
        s["prefix_len"] = ints(_history(c))
        cap = (max(_history(c)) + n + 15) // 16 * 16
        s["cache"] = _cache((B, cap), c["q8"], g, dev)
        s["row_offset"] = ints([_tree_parents(n, gc)[1] for _ in range(B)]) if c["tree"] else None
        s["n_rows"] = ints(_counts(c)) if c["ragged"] else None
    elif c["op"] == "attn":
        H = c["H"]
        cap = (c["hi"] + n + 15) // 16 * 16
        s["Q"] = torch.randn((B, H, n, DK), generator=g, device=dev).bfloat16()
        s["cache"] = _cache((B, cap), c["q8"], g, dev)
        s["prefix_len"] = ints(_history(c))
        s["mask"] = None
        if c["tree"]:
            m = torch.zeros((B, n, n), dtype=torch.uint8)
            for b in range(B):
                parent = _tree_parents(n, gc)[0]
                for i in range(n):
                    if i:
                        m[b, i] = m[b, parent[i]]
                    m[b, i, i] = 1
            s["mask"] = m.to(dev)
    elif c["op"] == "commit":
        cap = (max(_history(c)) + n + 15) // 16 * 16
        s["caches"] = _cache((c["layers"], B, cap), c["q8"], g, dev)
        s["prefix_len"] = ints(_history(c))
        s["n_accepted"] = ints(_accepted(c))
        # increasing node ids, the accepted ones first: a random choice of the tree's nodes
        path = [[-1] * n for _ in range(B)]
        for b, k in enumerate(_accepted(c)):
            path[b][:k] = sorted((1 + torch.randperm(n - 1, generator=gc)[:k]).tolist())
        s["path"] = ints(path)
    elif c["op"] == "read":
        cap = (max(_history(c)) + n + 15) // 16 * 16
        s["cache"] = _cache((B, cap), c["q8"], g, dev)
        s["first"] = ints(_history(c))
        s["n_rows"] = ints(_counts(c)) if c["ragged"] else None
        s["rows"] = torch.zeros((B, n, DK), dtype=torch.bfloat16, device=dev)
    else:
        H = c["H"]
        L = c["hi"] + n
        s["Q"] = torch.randn((B, n, H, NOPE + DR), generator=g, device=dev).bfloat16()
        # one product of the rows gives a head's 128 key values and its 128 values
        kv = torch.randn((B, L, H, NOPE + DV), generator=g, device=dev).bfloat16()
        s["K"], s["V"] = kv[..., :NOPE], kv[..., NOPE:]
        # the shared key where it stands, behind the latent vector in rows of 576
        s["K_rope"] = torch.randn((B, L, DK), generator=g, device=dev).bfloat16()[..., DC:]
        s["prefix_len"] = ints(_history(c))
        s["n_rows"] = ints(_counts(c)) if c["ragged"] else None
        s["O"] = torch.zeros((B, n, H, DV), dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.zeros((B, H, n), dtype=torch.float32, device=dev)
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _parts(cache):
    """The codes, rope keys and scales of 8-bit rows, as views."""
    return (cache[..., :DC].view(torch.float8_e4m3fn),
            cache[..., DC:DC + 2 * DR].view(torch.bfloat16),
            cache[..., DC + 2 * DR:].view(torch.float32))


def _values(rows):
    """fp32 rows [..., 576] of cache rows."""
    if rows.dtype != torch.uint8:
        return rows.float()
    code, rope, scale = _parts(rows)
    x = code.float().unflatten(-1, (DC // GROUP, GROUP)) * scale[..., None]
    return torch.cat([x.flatten(-2), rope.float()], -1)


def _held(cache):
    """A cache as outputs: 8-bit rows by their parts."""
    return _parts(cache) if cache.dtype == torch.uint8 else cache


def _plain_turn(x, cos, sin, interleaved):
    x = x.float()
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    a, b = x[..., :DR // 2], x[..., DR // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_append(s):
    c = s["case"]
    n = c["n"]
    i = torch.arange(n, device="cuda")
    off = i[None] if s["row_offset"] is None else s["row_offset"]
    pos = s["prefix_len"][:, None].double() + off.double()
    ang = pos[..., None] * s["inv_freq"].double()
    cos, sin = ang.cos().float(), ang.sin().float()
    got = (i[None] < (n if s["n_rows"] is None else s["n_rows"][:, None])).expand(c["B"], n)
    q = _plain_turn(s["q"], cos[:, :, None], sin[:, :, None], c["interleaved"]).bfloat16()
    s["q_out"].copy_(torch.where(got[..., None, None], q, s["q_out"]))
    x = s["kv"][..., :DC].float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
    r = _plain_turn(s["kv"][..., DC:], cos, sin, c["interleaved"])
    new = _pack(x, r) if c["q8"] else torch.cat([x, r], -1).bfloat16()
    at = (torch.arange(c["B"], device="cuda")[:, None], s["prefix_len"][:, None] + i[None])
    s["cache"][at] = torch.where(got[..., None], new, s["cache"][at])
    return s["q_out"], _held(s["cache"])


def _softmax_parts(x):
    """exp(x - max), its sum and log-sum-exp along the last axis; rows of -inf give zeros."""
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total > 0, total, torch.ones_like(total)), (top + total.log())[..., 0]


def _plain_attn(s):
    c = s["case"]
    B, n, H = c["B"], c["n"], c["H"]
    keys = _values(s["cache"])
    cap = keys.shape[1]
    x = (s["Q"].float().view(B, H * n, DK) @ keys.transpose(1, 2)).view(B, H, n, cap) * SCALE
    node = torch.arange(n, device="cuda")
    seen = s["mask"].bool() if s["mask"] is not None else (node[None, :] <= node[:, None])[None]
    seen = seen.expand(B, n, n)
    j = torch.arange(cap, device="cuda")[None] - s["prefix_len"][:, None]
    spec = seen.gather(2, j.clamp(0, n - 1)[:, None].expand(B, n, cap))
    see = (j < 0)[:, None] | ((j >= 0) & (j < n))[:, None] & spec
    p, lse = _softmax_parts(torch.where(see[:, None], x, -math.inf))
    o = p.view(B, H * n, cap) @ keys[..., :DC]
    return o.view(B, H, n, DC).bfloat16(), lse


def _plain_commit(s):
    c = s["case"]
    B, n = c["B"], c["n"]
    b = torch.arange(B, device="cuda")[:, None]
    k = torch.arange(n, device="cuda")[None]
    kept = k < s["n_accepted"][:, None]
    dst = (s["prefix_len"][:, None] + 1 + k).clamp(max=s["caches"].shape[2] - 1)
    src = torch.where(kept, s["prefix_len"][:, None] + s["path"], dst)
    # rows past the accepted ones keep what they hold (their index may be clamped: the last row)
    x = s["caches"]
    x[:, b, dst] = x[:, b, src]
    return _held(x)


def _plain_read(s):
    n = s["case"]["n"]
    i = torch.arange(n, device="cuda")[None]
    b = torch.arange(s["case"]["B"], device="cuda")[:, None]
    x = _values(s["cache"][b, s["first"][:, None] + i]).bfloat16()
    got = i < (n if s["n_rows"] is None else s["n_rows"][:, None])
    s["rows"].copy_(torch.where(got[..., None], x, s["rows"]))
    return s["rows"]


def _plain_prefill(s):
    c = s["case"]
    n = c["n"]
    q = s["Q"].float().transpose(1, 2)                                  # [B, H, n, 192]
    k, v = s["K"].float().permute(0, 2, 3, 1), s["V"].float().transpose(1, 2)
    x = q[..., :NOPE] @ k + q[..., NOPE:] @ s["K_rope"].float().transpose(1, 2)[:, None]
    i = torch.arange(n, device="cuda")
    j = torch.arange(k.shape[-1], device="cuda")
    see = j[None, None] <= s["prefix_len"][:, None, None] + i[None, :, None]
    p, lse = _softmax_parts(torch.where(see[:, None], x * SCALE, -math.inf))
    o = (p @ v).transpose(1, 2).bfloat16()
    got = i[None] < (n if s["n_rows"] is None else s["n_rows"][:, None])
    s["O"].copy_(torch.where(got[..., None, None], o, s["O"]))
    s["lse"].copy_(torch.where(got[:, None], lse, s["lse"]))
    return s["O"], s["lse"]


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------

def _own_append(s):
    from long_context_speculative_gb300 import rapid
    rapid.latent_append(s["kv"], s["cache"], s["prefix_len"], s["inv_freq"], q=s["q"],
                        q_out=s["q_out"], kv_weight=s["weight"], eps=EPS,
                        interleaved=s["case"]["interleaved"], row_offset=s["row_offset"],
                        n_rows=s["n_rows"])
    return s["q_out"], _held(s["cache"])


def _own_attn(s):
    from long_context_speculative_gb300 import rapid
    return rapid.latent_attn(s["Q"], s["cache"], s["prefix_len"], s["mask"], SCALE)


def _own_commit(s):
    from long_context_speculative_gb300 import rapid
    if "table" not in s:   # made once for a set of caches
        s["table"] = rapid.LatentLayerTable(list(s["caches"]))
    s["table"].commit(s["prefix_len"], s["path"], s["n_accepted"])
    return _held(s["caches"])


def _own_read(s):
    from long_context_speculative_gb300 import rapid
    return rapid.latent_read(s["cache"], s["first"], s["case"]["n"], n_rows=s["n_rows"],
                             out=s["rows"])


def _own_prefill(s):
    from long_context_speculative_gb300 import rapid
    return rapid.latent_prefill_attn(s["Q"], s["K"], s["V"], s["K_rope"], s["prefix_len"],
                                     n_rows=s["n_rows"], softmax_scale=SCALE, out=s["O"],
                                     lse=s["lse"])


def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "attn": _own_attn, "commit": _own_commit,
                "read": _own_read, "prefill": _own_prefill}[op](state)
    return {"append": _plain_append, "attn": _plain_attn, "commit": _plain_commit,
            "read": _plain_read, "prefill": _plain_prefill}[op](state)


# ---------------------------------------------------------------------------
# Definitions in 64 bits
# ---------------------------------------------------------------------------

def _e4m3(x):
    """Nearest e4m3 values (ties to the even last bit) of |x| <= 448, in 64 bits."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _exact_rows(cache):
    """Rows in 64 bits."""
    if cache.dtype != torch.uint8:
        return cache.double()
    code, rope, scale = _parts(cache)
    wide = scale.double().repeat_interleave(GROUP, -1)
    return torch.cat([code.double() * wide, rope.double()], -1)


def _exact_held(cache):
    return tuple(x.double() for x in _parts(cache)) if cache.dtype == torch.uint8 else cache.double()


def _exact_append(s):
    c = s["case"]
    h = DR // 2
    q_out = s["q_out"].double()
    held = _exact_held(s["cache"])
    first, second = ((slice(0, DR, 2), slice(1, DR, 2)) if c["interleaved"]
                     else (slice(0, h), slice(h, DR)))
    for b, m in enumerate(_counts(c)):
        p0 = int(s["prefix_len"][b])
        steps = torch.arange(m, device="cuda") if s["row_offset"] is None else s["row_offset"][b, :m]
        # the rotation as one complex factor per pair
        turn = torch.polar(torch.ones((m, h), dtype=torch.float64, device="cuda"),
                           torch.outer(steps.double() + p0, s["inv_freq"].double()))

        def turned(x, f):
            z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * f
            y = torch.empty_like(x)
            y[..., first], y[..., second] = z.real, z.imag
            return y

        q_out[b, :m] = turned(s["q"][b, :m].double(), turn[:, None])
        row = s["kv"][b, :m].double()
        x = row[:, :DC]
        x = x / (x.pow(2).sum(-1, keepdim=True) / DC + EPS).sqrt() * s["weight"].double()
        r = turned(row[:, DC:], turn)
        at = slice(p0, p0 + m)
        if not c["q8"]:
            held[b, at] = torch.cat([x, r], -1)
            continue
        for k in range(DC // GROUP):
            y = x[:, k * GROUP:(k + 1) * GROUP]
            top = y.abs().amax(-1) / E4M3_MAX
            near = torch.exp2(torch.ceil(torch.log2(top.clamp(min=2.0 ** SCALE_EXP_MIN))))
            # log2 of a power of two may land beside the whole number
            near = torch.where((top <= near / 2) & (near > 2.0 ** SCALE_EXP_MIN), near / 2, near)
            near = torch.where(top > 0, near, torch.ones_like(near))
            held[0][b, at, k * GROUP:(k + 1) * GROUP] = _e4m3(y / near[:, None])
            held[2][b, at, k] = near
        held[1][b, at] = r
    return q_out, held


def _exact_attn(s):
    c = s["case"]
    B, n, H = c["B"], c["n"], c["H"]
    O = torch.zeros((B, H, n, DC), dtype=torch.float64, device="cuda")
    lse = torch.zeros((B, H, n), dtype=torch.float64, device="cuda")
    for b, P in enumerate(_history(c)):
        rows = _exact_rows(s["cache"][b, :P + n])
        hidden = torch.zeros((n, P + n), dtype=torch.bool, device="cuda")
        tree = s["mask"][b] if s["mask"] is not None else torch.ones((n, n), device="cuda").tril()
        hidden[:, P:] = tree == 0
        for h in range(0, H, 16):
            q = s["Q"][b, h:h + 16].double()
            x = (torch.einsum("hid,jd->hij", q, rows) * SCALE).masked_fill(hidden, -math.inf)
            lse[b, h:h + 16] = torch.logsumexp(x, -1)
            O[b, h:h + 16] = torch.softmax(x, -1) @ rows[:, :DC]
    return O, lse


def _exact_commit(s):
    x = s["caches"].clone()
    path = s["path"].tolist()
    for b, k in enumerate(_accepted(s["case"])):
        P = int(s["prefix_len"][b])
        x[:, b, P + 1:P + 1 + k] = s["caches"][:, b, [P + i for i in path[b][:k]]]
    return _exact_held(x)


def _exact_read(s):
    out = s["rows"].double()
    for b, m in enumerate(_counts(s["case"])):
        p0 = int(s["first"][b])
        out[b, :m] = _exact_rows(s["cache"][b, p0:p0 + m])
    return out


def _exact_prefill(s):
    c = s["case"]
    O, lse = s["O"].double(), s["lse"].double()
    for b, (P, m) in enumerate(zip(_history(c), _counts(c))):
        later = torch.ones((m, P + m), dtype=torch.bool, device="cuda").triu(P + 1)
        for h in range(c["H"]):
            keys = torch.cat([s["K"][b, :P + m, h], s["K_rope"][b, :P + m]], -1).double()
            x = (s["Q"][b, :m, h].double() @ keys.T * SCALE).masked_fill(later, -math.inf)
            lse[b, h, :m] = torch.logsumexp(x, -1)
            O[b, :m, h] = torch.softmax(x, -1) @ s["V"][b, :P + m, h].double()
    return O, lse


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attn": _exact_attn, "commit": _exact_commit,
            "read": _exact_read, "prefill": _exact_prefill}[case["op"]](s)


# ---------------------------------------------------------------------------
# Bytes and operations that the path cannot do without
# ---------------------------------------------------------------------------

def work(case):
    c = case
    row = ROW_BYTES if c.get("q8") else 2 * DK
    if c["op"] == "append":
        m = sum(_counts(c))
        return {"bytes": float(m * (2 * 2 * c["H"] * DR + 2 * DK + row) + 2 * DC + 2 * DR),
                "flops": float(m * (3 * DR * (c["H"] + 1) + 4 * DC))}
    if c["op"] == "attn":
        keys = sum(P + c["n"] for P in _history(c))
        rows = c["H"] * c["n"]
        return {"bytes": float(keys * row + c["B"] * rows * (2 * DK + 2 * DC + 4)),
                "flops": 2.0 * rows * keys * (DK + DC)}
    if c["op"] == "commit":
        return {"bytes": 2.0 * c["layers"] * sum(_accepted(c)) * row, "flops": 0.0}
    if c["op"] == "read":
        m = sum(_counts(c))
        return {"bytes": float(m * (row + 2 * DK)), "flops": float(m * DC if c["q8"] else 0)}
    bytes_, pairs = 0.0, 0.0
    for P, m in zip(_history(c), _counts(c)):
        pairs += m * P + m * (m + 1) / 2
        bytes_ += 2 * m * c["H"] * (NOPE + DR + DV) + 4 * m * c["H"]
        bytes_ += 2 * (P + m) * (c["H"] * (NOPE + DV) + DR)
    return {"bytes": bytes_, "flops": 2.0 * c["H"] * pairs * (NOPE + DR + DV)}
