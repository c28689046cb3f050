"""Cases of the serving operators around an 8-bit key/value cache, with their plain forms.

Three operators form the path of one verify step over a history held in 8 bits:

* ``append``  the projections' rows of a step or a prefill chunk: queries and keys get
              their norm for each head and the rotation by position, keys and values go
              into the cache's 16-bit (or 32-bit) tail, queries into the layout that
              attention reads (``rapid.qkv_append``);
* ``seal``    whole blocks of 64 committed tail rows move into pages of 8-bit values
              with one scale for each block, head and side, on every layer
              (``rapid.Q8LayerTable.seal``);
* ``attn``    attention of the verify queries over the pages, the tail and the
              speculative rows (``rapid.verify_attn_q8``).

``run`` takes a state from ``prepare`` through one of them: with ``own`` false as
elementary torch operations in 32 bits, with ``own`` true as the library's calls.
``exact`` gives the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

BLOCK = 64          # tokens of a page
E4M3_MAX = 448.0
THETA = 500000.0
EPS = 1e-5
SCALE_EXP_MIN = -64  # smallest exponent of a block's scale

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _append(name, B, n, Hq, Hkv, d, dtype, norm, rot, interleaved=False, tree=False, ragged=False,
            base=0):
    return dict(name=name, op="append", B=B, n=n, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, norm=norm,
                rot=rot, interleaved=interleaved, tree=tree, ragged=ragged, base=base)


def _seal(name, layers, B, Hkv, d, dtype, tail, keep):
    return dict(name=name, op="seal", layers=layers, B=B, Hkv=Hkv, d=d, dtype=dtype, tail=tail,
                keep=keep)


def _attn(name, B, n, Hq, Hkv, d, dtype, lo, hi, tail, tree=False):
    return dict(name=name, op="attn", B=B, n=n, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, lo=lo, hi=hi,
                tail=tail, tree=tree)


def listed():
    return [
        # one verify step of an 11-node chain (Llama-3.1-8B shape) at a position far into a
        # 120K context: a call of a few microseconds between two matrix products
        _append("append_step_8b", 1, 11, 32, 8, 128, "bf16", False, 128, base=122880),
        # a prefill chunk of the same shape, with query and key norms: bandwidth counts
        _append("append_prefill_8b", 1, 8192, 32, 8, 128, "bf16", True, 128, base=65536),
        # sequences of different chunk lengths, 32-bit tensors, head dimension 64, half of
        # each head rotated in interleaved pairs
        _append("append_ragged_f32_d64", 3, 1999, 32, 8, 64, "f32", True, 32, interleaved=True,
                ragged=True, base=1021),
        # after a step: one block or none of each of four sequences is full, 32 layers
        _seal("seal_step_32layers", 32, 4, 8, 128, "bf16", 75, 0),
        # after a prefill chunk of about 2K tokens: 33 blocks of every layer and head
        _seal("seal_prefill_32layers", 32, 1, 8, 128, "bf16", 2131, 11),
        # the tiny 32-bit shape: 4 heads over one KV head, about 1K tokens of history
        _attn("attn_tiny_f32", 1, 5, 4, 1, 64, "f32", 16, 16, 5),
        # one token of plain decode over a short history: latency
        _attn("attn_decode_4k_8b", 1, 1, 32, 8, 128, "bf16", 64, 64, 13),
        # the 11-node chain at 32K and 120K (Llama-3.1-8B shape)
        _attn("attn_chain_32k_8b", 1, 11, 32, 8, 128, "bf16", 511, 511, 53),
        _attn("attn_chain_120k_8b", 1, 11, 32, 8, 128, "bf16", 1919, 1919, 59),
        # the same chain on the Llama-3.1-70B shape at 128K: 88 rows to a KV head
        _attn("attn_chain_128k_70b", 1, 11, 64, 8, 128, "bf16", 2047, 2047, 37),
        # a tree of 32 nodes on four ragged histories of 32K to 96K (Qwen2.5-7B shape)
        _attn("attn_tree_ragged_7b", 4, 32, 28, 4, 128, "bf16", 512, 1535, 61, tree=True),
        # head dimension 64 (Llama-3.2-1B shape) at 120K
        _attn("attn_chain_120k_d64", 1, 11, 32, 8, 64, "bf16", 1919, 1919, 23),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "seal", "attn", "attn"])
    Hq, Hkv = rng.choice([(32, 8), (64, 8), (28, 4), (14, 2), (16, 16), (4, 1)])
    d = rng.choice([64, 128])
    if op == "append":
        B = rng.randint(1, 6)
        tree = rng.random() < 0.3
        n = rng.randint(1, 64) if tree else _log_int(rng, 1, 8192 * 40 * 128 // (B * (Hq + Hkv) * d))
        rot = rng.choice([16, 32, d // 2, d, d])
        c = _append("", B, n, Hq, Hkv, d, rng.choice(["bf16", "bf16", "f32"]),
                    rng.random() < 0.6, rot, rng.random() < 0.3, tree, rng.random() < 0.4,
                    _log_int(rng, 1, 1 << 20))
        if c["dtype"] == "f32":
            c["n"] = max(1, c["n"] // 2)
    elif op == "seal":
        layers, B = _log_int(rng, 1, 64), rng.randint(1, 6)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        most = 32 * 8 * 2100 * 128 // (layers * B * Hkv * d * (1 if dtype == "bf16" else 2))
        tail = _log_int(rng, 64, max(65, min(8192, most)))
        c = _seal("", layers, B, Hkv, d, dtype, tail, rng.choice([0, rng.randint(0, tail - 64)]))
    else:
        B = rng.randint(1, 6)
        n = rng.choice([1, rng.randint(2, 16), rng.randint(2, 16), rng.randint(17, 64)])
        rows = (Hq // Hkv) * n
        most = max(1, min(2048 * 8 // (B * Hkv), 4096 * 224 * 16 // (rows * B * Hkv)))
        dtype = "f32" if rng.random() < 0.15 else "bf16"
        if dtype == "f32":
            most = max(1, min(most, 4096 // (rows * B)))
        hi = _log_int(rng, 1, most)
        lo = hi if rng.random() < 0.4 else rng.randint(0, hi)
        c = _attn("", B, n, Hq, Hkv, d, dtype, lo, hi, rng.randint(0, 127), rng.random() < 0.4)
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# Lengths of a case's sequences (the case alone decides them)
# ---------------------------------------------------------------------------

def _blocks(c):
    """Sealed blocks of each sequence: from lo to hi, the odd ones among them."""
    B, lo, hi = c["B"], c["lo"], c["hi"]
    return [hi] if B == 1 else [lo + (hi - lo) * b // (B - 1) for b in range(B)]


def _tails(c):
    """Tail rows of each sequence."""
    return [max(0, c["tail"] - 17 * b) for b in range(c["B"])]


def _tail_cap(c):
    n = c["n"] if c["op"] == "attn" else 11
    return (c["tail"] + n + 15) // 16 * 16


def _counts(c):
    """Rows that each sequence appends."""
    return [c["n"] if not c["ragged"] else max(1, c["n"] - (c["n"] * b) // (c["B"] + 1))
            for b in range(c["B"])]


def _sealed_now(c):
    return [max(0, t - c["keep"]) // BLOCK for t in _tails(c)]


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _tree_parents(n, g):
    """Parents of a random tree of depth up to 6 below the root."""
    parent, depth = [-1], [0]
    for i in range(1, n):
        free = [j for j in range(i) if depth[j] < 6]
        j = free[int(torch.randint(len(free), (1,), generator=g))]
        parent.append(j)
        depth.append(depth[j] + 1)
    return parent, depth


def _block_scale(amax):
    """The power of two that brings amax into e4m3's range (1 for an all-zero block)."""
    m, e = torch.frexp(amax)
    e = e - 9 + (m > 0.875).to(e.dtype)   # 448 = 0.875 * 2^9
    e = torch.where(amax > 0, e.clamp(min=SCALE_EXP_MIN), torch.zeros_like(e))
    return torch.ldexp(torch.ones_like(amax), e)


def _rows(shape, g, dtype, dev):
    """Rows as projections give them: a spread of sizes over the channels."""
    x = torch.randn(shape, generator=g, device=dev)
    x *= torch.exp(0.5 * torch.randn(shape[-1:], generator=g, device=dev))
    return x.to(dtype)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    gc = torch.Generator().manual_seed(seed)
    c, s = case, {"case": case}
    dt, B, Hkv, d = DT[c["dtype"]], c["B"], c["Hkv"], c["d"]

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    if c["op"] == "append":
        Hq, n = c["Hq"], c["n"]
        # one fused projection: a row holds all query heads, then keys, then values
        qkv = _rows((B, n, Hq + 2 * Hkv, d), g, dt, dev)
        s["q"], s["k"], s["v"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
        cap = (n + 64 + 15) // 16 * 16
        s["K"], s["V"] = _rows((B, Hkv, cap, d), g, dt, dev), _rows((B, Hkv, cap, d), g, dt, dev)
        s["Q"] = torch.zeros((B, Hq, n, d), dtype=dt, device=dev)
        s["prefix_len"] = ints([(37 + 11 * b) % 64 for b in range(B)])
        s["pos_offset"] = ints([c["base"] + 64 * b for b in range(B)])
        s["inv_freq"] = THETA ** (-torch.arange(0, c["rot"], 2, device=dev).double() / c["rot"])
        s["inv_freq"] = s["inv_freq"].float()
        s["q_weight"] = s["k_weight"] = None
        if c["norm"]:
            s["q_weight"] = (1 + 0.2 * torch.randn(d, generator=g, device=dev)).to(dt)
            s["k_weight"] = (1 + 0.2 * torch.randn(d, generator=g, device=dev)).to(dt)
        s["row_offset"] = None
        if c["tree"]:
            s["row_offset"] = ints([_tree_parents(n, gc)[1] for _ in range(B)])
        s["n_rows"] = ints(_counts(c)) if c["ragged"] else None
    elif c["op"] == "seal":
        L, cap, n_b = c["layers"], _tail_cap(c), _sealed_now(c)
        s["K"] = _rows((L, B, Hkv, cap, d), g, dt, dev)
        s["V"] = _rows((L, B, Hkv, cap, d), g, dt, dev)
        before = [3 + b for b in range(B)]            # blocks sealed earlier
        per = max(x + y for x, y in zip(before, n_b)) + 1
        pages = B * per
        s["pages"] = torch.zeros((L, pages, Hkv, 2, BLOCK, d), dtype=torch.float8_e4m3fn, device=dev)
        s["scales"] = torch.ones((L, pages, Hkv, 2), device=dev)
        s["page_table"] = torch.randperm(pages, generator=gc).to(torch.int32).view(B, per).to(dev)
        s["sealed_len"] = ints([BLOCK * x for x in before])
        s["tail_len"] = ints(_tails(c))
    else:
        Hq, n, blocks = c["Hq"], c["n"], _blocks(c)
        per = max(1, max(blocks))
        pages = B * per + 1
        cap = _tail_cap(c)
        s["Q"] = torch.randn((B, Hq, n, d), generator=g, device=dev).to(dt)
        s["K"], s["V"] = _rows((B, Hkv, cap, d), g, dt, dev), _rows((B, Hkv, cap, d), g, dt, dev)
        raw = _rows((pages, Hkv, 2, BLOCK, d), g, torch.float32, dev)
        s["scales"] = _block_scale(raw.abs().amax(dim=(3, 4)))
        s["pages"] = (raw / s["scales"][..., None, None]).to(torch.float8_e4m3fn)
        # pages of the sequences in the order in which a serving pool handed them out
        s["page_table"] = torch.randperm(pages, generator=gc)[:B * per].to(torch.int32).view(B, per)
        s["page_table"] = s["page_table"].to(dev)
        s["sealed_len"] = ints([BLOCK * x for x in blocks])
        s["tail_len"] = ints(_tails(c))
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
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _plain_head(x, weight, cos, sin, c):
    """Norm and rotation of rows [B, n, H, d] in 32 bits."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    rot = c["rot"]
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_append(s):
    c = s["case"]
    n, dt = c["n"], DT[c["dtype"]]
    i = torch.arange(n, device="cuda")
    off = i[None] if s["row_offset"] is None else s["row_offset"]
    pos = (s["prefix_len"] + s["pos_offset"])[:, None].double() + off.double()
    ang = pos[..., None] * s["inv_freq"].double()
    cos, sin = ang.cos().float()[:, :, None], ang.sin().float()[:, :, None]
    q = _plain_head(s["q"], s["q_weight"], cos, sin, c).to(dt).transpose(1, 2)
    k = _plain_head(s["k"], s["k_weight"], cos, sin, c).to(dt).transpose(1, 2)
    v = s["v"].transpose(1, 2)
    count = n if s["n_rows"] is None else s["n_rows"][:, None]
    s["Q"].copy_(torch.where((i[None] < count)[:, None, :, None], q, s["Q"]))
    at = torch.arange(s["K"].shape[2], device="cuda")[None] - s["prefix_len"][:, None]
    new = ((at >= 0) & (at < count))[:, None, :, None]
    at = at.clamp(0, n - 1)[:, None, :, None].expand(s["K"].shape).long()
    s["K"].copy_(torch.where(new, k.gather(2, at), s["K"]))
    s["V"].copy_(torch.where(new, v.gather(2, at), s["V"]))
    return s["Q"], s["K"], s["V"]


def _plain_seal(s):
    c = s["case"]
    L, B, Hkv, cap, d = s["K"].shape
    most = cap // BLOCK
    n_b = (s["tail_len"] - c["keep"]).clamp(min=0) // BLOCK
    x = torch.stack([s["K"], s["V"]], 3)[..., :most * BLOCK, :].float()
    x = x.view(L, B, Hkv, 2, most, BLOCK, d).permute(0, 1, 4, 2, 3, 5, 6)
    x = x.reshape(L, B * most, Hkv, 2, BLOCK, d)
    scale = _block_scale(x.abs().amax(dim=(-1, -2)))
    code = (x / scale[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    # which block goes to which page: the pool's extra last entry takes the blocks that stay
    pages = s["pages"].shape[1]
    j = torch.arange(most, device="cuda")[None]
    slot = (s["sealed_len"][:, None] // BLOCK + j).clamp(max=s["page_table"].shape[1] - 1)
    page = torch.where(j < n_b[:, None], s["page_table"].gather(1, slot.long()).long(), pages)
    src = torch.full((pages + 1,), -1, device="cuda")
    src[page.flatten()] = torch.arange(B * most, device="cuda")
    src = src[:pages]
    got = (src >= 0)[None, :, None, None]
    s["scales"].copy_(torch.where(got, scale[:, src.clamp(min=0)], s["scales"]))
    old = s["pages"].view(torch.uint8)
    old.copy_(torch.where(got[..., None, None], code[:, src.clamp(min=0)], old))
    # the rows that stay move to the front
    r = torch.arange(cap, device="cuda")[None]
    moved = BLOCK * n_b[:, None]
    here = ((r < s["tail_len"][:, None] - moved) & (moved > 0))[None, :, None, :, None]
    at = (r + moved).clamp(max=cap - 1)[None, :, None, :, None].expand(s["K"].shape).long()
    for t in (s["K"], s["V"]):
        t.copy_(torch.where(here, t.gather(3, at), t))
    return s["pages"], s["scales"], s["K"], s["V"]


def _plain_attn(s):
    c = s["case"]
    B, n, Hq, Hkv, d = c["B"], c["n"], c["Hq"], c["Hkv"], c["d"]
    at = s["page_table"].long()
    kv = s["pages"][at].float() * s["scales"][at][..., None, None]   # [B, blocks, Hkv, 2, 64, d]
    kv = kv.permute(3, 0, 2, 1, 4, 5).reshape(2, B, Hkv, -1, d)
    sealed, cap = kv.shape[3], s["K"].shape[2]
    q = s["Q"].float().view(B, Hkv, -1, d)
    x = torch.cat([q @ kv[0].transpose(2, 3), q @ s["K"].float().transpose(2, 3)], 3)
    x = x.view(B, Hkv, Hq // Hkv, n, -1) / math.sqrt(d)
    node = torch.arange(n, device="cuda")
    seen = s["mask"].bool() if s["mask"] is not None else (node[None, :] <= node[:, None])[None]
    seen = seen.expand(B, n, n)
    j = torch.arange(cap, device="cuda")[None] - s["tail_len"][:, None]
    spec = seen.gather(2, j.clamp(0, n - 1)[:, None].expand(B, n, cap))
    tail = (j < 0)[:, None] | ((j >= 0) & (j < n))[:, None] & spec
    pages = torch.arange(sealed, device="cuda")[None, None] < s["sealed_len"][:, None, None]
    seen = torch.cat([pages.expand(B, n, sealed), tail], 2)[:, None, None]
    x = torch.where(seen, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    lse = (top + total.log()).view(B, Hq, n)
    p = (p / torch.where(total > 0, total, torch.ones_like(total))).view(B, Hkv, q.shape[2], -1)
    o = p[..., :sealed] @ kv[1] + p[..., sealed:] @ s["V"].float()
    return o.view(B, Hq, n, d).to(DT[c["dtype"]]), lse


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------

def _own_append(s):
    from long_context_speculative_gb300 import rapid
    rapid.qkv_append(s["q"], s["k"], s["v"], s["K"], s["V"], s["prefix_len"], s["inv_freq"],
                     q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                     interleaved=s["case"]["interleaved"], pos_offset=s["pos_offset"],
                     row_offset=s["row_offset"], n_rows=s["n_rows"], out=s["Q"])
    return s["Q"], s["K"], s["V"]


def _own_seal(s):
    from long_context_speculative_gb300 import rapid
    if "table" not in s:   # made once for a set of caches, as for rapid_kv_commit
        s["table"] = rapid.Q8LayerTable(list(s["K"]), list(s["V"]), list(s["pages"]),
                                        list(s["scales"]))
    s["table"].seal(s["page_table"], s["sealed_len"], s["tail_len"], s["case"]["keep"])
    return s["pages"], s["scales"], s["K"], s["V"]


def _own_attn(s):
    from long_context_speculative_gb300 import rapid
    return rapid.verify_attn_q8(s["Q"], s["K"], s["V"], s["pages"], s["scales"], s["page_table"],
                                s["sealed_len"], s["tail_len"], s["mask"])


def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "seal": _own_seal, "attn": _own_attn}[op](state)
    return {"append": _plain_append, "seal": _plain_seal, "attn": _plain_attn}[op](state)


# ---------------------------------------------------------------------------
# Definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_append(s):
    c = s["case"]
    n, d, rot, h = c["n"], c["d"], c["rot"], c["rot"] // 2
    Q, K, V = s["Q"].double(), s["K"].double(), s["V"].double()
    counts = _counts(c)
    # the rotation as one complex factor per pair
    first, second = ((slice(0, rot, 2), slice(1, rot, 2)) if c["interleaved"]
                     else (slice(0, h), slice(h, rot)))
    for b in range(c["B"]):
        m, p0 = counts[b], int(s["prefix_len"][b])
        steps = torch.arange(m, device="cuda") if s["row_offset"] is None else s["row_offset"][b, :m]
        pos = steps.double() + (p0 + int(s["pos_offset"][b]))
        turn = torch.polar(torch.ones((m, h), dtype=torch.float64, device="cuda"),
                           torch.outer(pos, s["inv_freq"].double()))[:, None]
        for x, w, out in ((s["q"], s["q_weight"], "q"), (s["k"], s["k_weight"], "k")):
            y = x[b, :m].double()
            if w is not None:
                y = y / (y.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt() * w.double()
            z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * turn
            y[..., first], y[..., second] = z.real, z.imag
            if out == "q":
                Q[b, :, :m] = y.transpose(0, 1)
            else:
                K[b, :, p0:p0 + m] = y.transpose(0, 1)
        V[b, :, p0:p0 + m] = s["v"][b, :m].double().transpose(0, 1)
    return Q, K, V


def _e4m3(x):
    """Nearest e4m3 values (ties to the even last bit) of |x| <= 448, in 64 bits."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _exact_seal(s):
    c = s["case"]
    pages, scales = s["pages"].double(), s["scales"].double()
    K, V = s["K"].double(), s["V"].double()
    for b, n_b in enumerate(_sealed_now(c)):
        first = int(s["sealed_len"][b]) // BLOCK
        for j in range(n_b):
            page = int(s["page_table"][b, first + j])
            for side, t in enumerate((K, V)):
                x = t[:, b, :, j * BLOCK:(j + 1) * BLOCK]
                top = x.abs().amax(dim=(2, 3)) / E4M3_MAX
                near = torch.exp2(torch.ceil(torch.log2(top.clamp(min=2.0 ** SCALE_EXP_MIN))))
                # log2 of a power of two may land beside the whole number
                scale = torch.where((top <= near / 2) & (near > 2.0 ** SCALE_EXP_MIN), near / 2, near)
                scale = torch.where(top > 0, scale, torch.ones_like(top))
                scales[:, page, :, side] = scale
                pages[:, page, :, side] = _e4m3(x / scale[..., None, None])
        rest = _tails(c)[b] - n_b * BLOCK
        if n_b:
            for t in (K, V):
                t[:, b, :, :rest] = t[:, b, :, n_b * BLOCK:n_b * BLOCK + rest].clone()
    return pages, scales, K, V


def _exact_attn(s):
    c = s["case"]
    n, G, d = c["n"], c["Hq"] // c["Hkv"], c["d"]
    O = torch.zeros(s["Q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["Q"].shape[:3], dtype=torch.float64, device="cuda")
    for b in range(c["B"]):
        ids = s["page_table"][b, :_blocks(c)[b]].long()
        t = _tails(c)[b]
        hidden = torch.zeros((n, len(ids) * BLOCK + t + n), dtype=torch.bool, device="cuda")
        tree = s["mask"][b] if s["mask"] is not None else torch.ones((n, n), device="cuda").tril()
        hidden[:, -n:] = tree == 0
        for g in range(c["Hkv"]):
            unit = s["scales"][ids, g].double()[..., None, None]
            both = s["pages"][ids, g].double() * unit
            keys = torch.cat([both[:, 0].reshape(-1, d), s["K"][b, g, :t + n].double()])
            vals = torch.cat([both[:, 1].reshape(-1, d), s["V"][b, g, :t + n].double()])
            for h in range(g * G, (g + 1) * G):
                x = (s["Q"][b, h].double() @ keys.T * d ** -0.5).masked_fill(hidden, -math.inf)
                lse[b, h] = torch.logsumexp(x, 1)
                O[b, h] = (x - lse[b, h, :, None]).exp() @ vals
    return O, lse


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "seal": _exact_seal, "attn": _exact_attn}[case["op"]](s)


# ---------------------------------------------------------------------------
# Bytes and operations that the path cannot do without
# ---------------------------------------------------------------------------

def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    d = c["d"]
    if c["op"] == "append":
        rows = sum(_counts(c))
        heads = c["Hq"] + 2 * c["Hkv"]
        turned = rows * (c["Hq"] + c["Hkv"])
        return {"bytes": 2.0 * rows * heads * d * e + 2 * c["rot"],
                "flops": float(turned * (3 * c["rot"] + (4 * d if c["norm"] else 0)))}
    if c["op"] == "seal":
        heads = 2 * c["layers"] * c["Hkv"]
        n_b = _sealed_now(c)
        sealed = sum(n_b) * BLOCK * d
        moved = sum((t - BLOCK * k) * d for t, k in zip(_tails(c), n_b) if k)
        return {"bytes": float(heads * (sealed * (e + 1) + 4 * sum(n_b) + 2 * e * moved)),
                "flops": 2.0 * heads * sealed}
    keys = sum(BLOCK * x for x in _blocks(c))
    tail = sum(t + c["n"] for t in _tails(c))
    rows = c["Hq"] * c["n"]
    return {"bytes": float(c["Hkv"] * 2 * (keys * d + keys // BLOCK * 4 + tail * d * e)
                           + c["B"] * rows * (2 * d * e + 4)),
            "flops": 4.0 * rows * d * (keys + tail)}
