"""Cases, plain forms and exact forms of the operators on an 8-bit KV cache.

The cache holds K, V and the index key as e4m3 codes with one fp32 scale for each
(block of tokens, KV head) (for the index key: each block), so that a value is
code * scale.  Four operators work on it:

  append  quantises new bf16 rows into the cache.  A block's scale is the smallest
          power of two that maps its largest finite magnitude into [-448, 448] (never
          below 2^-100); a block that holds older rows keeps the larger of its scale
          and the one the new rows need, and its older rows are rounded to it.
  read    gives rows of the cache back as bf16.
  scores  max over the visible tokens of a block of <q_idx, k_idx>, for every block.
  attn    softmax attention of every query head over the blocks its group selected.

``run`` computes them in elementary torch operations, or (``own``) calls the
framework.  ``exact`` states them in 64 bits.
"""

import torch

own = False

LARGEST = 448.0  # largest e4m3 value
LEAST = 2.0 ** -100  # smallest scale
F8 = torch.float8_e4m3fn
DEV = "cuda"


# ------------------------------------------------------------------ the cases
def _case(name, op, **kw):
    c = dict(name=name, op=op, batch=1, n=1, max_kv=1024, H=8, h=2, d=128, d_idx=128, block=64,
             topk=8, paged=False, ragged=False)
    c.update(kw)
    return c


def listed():
    return [
        # one decode step's cache write: a row a sequence, mostly launch latency
        _case("append_step", "append", batch=16, max_kv=2048, h=8),
        # a whole prompt written at once: bandwidth
        _case("append_prompt", "append", batch=2, n=32768, max_kv=32768, h=4, d_idx=64),
        # chunks of ragged sequences into small pages, blocks that are partly filled already
        _case("append_pages", "append", batch=3, n=301, max_kv=1500, h=2, d=64, d_idx=32, block=16,
              paged=True, ragged=True),
        # a prompt's cache taken out in bf16 (to move or inspect it)
        _case("read_prompt", "read", batch=2, n=32768, max_kv=32768, h=4, d_idx=64),
        # some rows of ragged sequences out of pages
        _case("read_pages", "read", batch=3, n=777, max_kv=1500, h=2, d=64, d_idx=32, block=32,
              paged=True, ragged=True),
        # the index scan of one decode step at 128K tokens
        _case("scores_step_128k", "scores", batch=16, max_kv=131072, h=8),
        # the same for a few short ragged sequences in pages
        _case("scores_step_ragged", "scores", batch=5, max_kv=999, h=3, d_idx=64, block=32,
              paged=True, ragged=True),
        # the index scores of a 2048-query chunk of a 32K prompt
        _case("scores_chunk_32k", "scores", n=2048, max_kv=32768, h=4, d_idx=64),
        # attention of one decode step at 128K tokens
        _case("attn_step_128k", "attn", batch=16, max_kv=131072, H=64, h=8, topk=128),
        # one token of one short sequence with small blocks: latency
        _case("attn_step_small", "attn", max_kv=900, H=6, h=2, d=64, block=16),
        # a 4096-query chunk of a 32K prompt
        _case("attn_chunk_32k", "attn", n=4096, max_kv=32768, H=32, h=4, topk=32),
        # ragged sequences in pages, some queries before their sequence's first token
        _case("attn_chunk_pages", "attn", batch=3, n=333, max_kv=700, H=20, h=2, d=64, block=32,
              paged=True, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(("append", "read", "scores", "attn"))
    h = rng.choice((1, 2, 3, 4, 8))
    c = dict(op=op, h=h, H=h * rng.randint(1, 16), d=rng.choice((64, 128)),
             d_idx=rng.choice((32, 64, 128)), block=rng.choice((16, 32, 64, 128)),
             paged=rng.random() < 0.5, ragged=rng.random() < 0.7, topk=1)
    if op in ("append", "read"):
        c["max_kv"] = _log(rng, 200, 30000)
        c["n"] = 1 if rng.random() < 0.4 else _log(rng, 2, c["max_kv"])
        c["batch"] = rng.randint(1, max(1, min(24, 60000 // c["max_kv"])))
    elif op == "scores":
        c["max_kv"] = _log(rng, 100, 60000)
        c["n"] = 1 if rng.random() < 0.6 else _log(rng, 2, min(1500, c["max_kv"]))
        c["batch"] = rng.randint(1, 12) if c["n"] == 1 else rng.randint(1, 2)
    else:
        c["max_kv"] = _log(rng, 100, 20000)
        c["n"] = 1 if rng.random() < 0.6 else _log(rng, 2, min(1000, c["max_kv"]))
        c["batch"] = rng.randint(1, 12) if c["n"] == 1 else rng.randint(1, 2)
        c["topk"] = _log(rng, 1, max(1, (8192 if c["n"] == 1 else 1024) // c["block"]))
    return c


def _blocks(c):
    return -(-c["max_kv"] // c["block"])


def work(c):
    """Bytes and operations of one pass (mean lengths where the sequences are ragged)."""
    b, n, h, d, di, B, H = c["batch"], c["n"], c["h"], c["d"], c["d_idx"], c["block"], c["H"]
    row = h * 2 * d + di  # codes of one token
    if c["op"] == "append":
        return {"bytes": b * n * row * 3 + b * (-(-n // B)) * (2 * h + 1) * 4, "flops": b * n * row}
    if c["op"] == "read":
        have = n / 2 if c["ragged"] else n
        return {"bytes": b * have * row * 3 + b * (-(-n // B)) * (2 * h + 1) * 4,
                "flops": b * have * row}
    length = c["max_kv"] / 2 if c["ragged"] else c["max_kv"]
    if c["op"] == "scores":
        seen = length - (0 if n == 1 else min(n, length) / 2)
        return {"bytes": b * (length * di + length / B * 4 + n * h * (di * 2 + _blocks(c) * 4)),
                "flops": 2.0 * b * n * h * di * seen}
    keys = min(c["topk"] * B, length - (0 if n == 1 else min(n, length) / 2))
    cache = min(n * keys, length) * h * (2 * d + 8 / B)
    return {"bytes": b * (cache + n * (H * (4 * d + 4) + h * c["topk"] * 4)),
            "flops": 4.0 * b * n * H * d * keys}


# ------------------------------------------------------------------ the inputs
def _scale_of(amax):
    """Smallest power of two s >= 2^-100 with amax <= 448 s."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [1/2, 1); 448 = 0.875 * 2^9
    s = torch.ldexp(torch.ones_like(amax), e - 9 + (m > 0.875).int())
    return torch.where(amax > 0, s, 0.0).clamp_min(LEAST)


def _codes(x, s):
    return (x / s).clamp(-LARGEST, LARGEST).to(F8)


def _filled(shape, blk, gen):
    """Codes [outer, tokens, d] and scales [outer, blocks] of normal rows whose size
    differs from block to block, as between heads and passages of a text."""
    outer, tokens, d = shape
    nblk = -(-tokens // blk)
    codes = torch.empty((outer, tokens, d), dtype=F8, device=DEV)
    scales = torch.empty((outer, nblk), device=DEV)
    step = max(1, (1 << 27) // (nblk * blk * d))
    for i in range(0, outer, step):
        k = min(step, outer - i)
        x = torch.randn((k, nblk, blk * d), device=DEV, generator=gen)
        x *= torch.exp2(torch.rand((k, nblk, 1), device=DEV, generator=gen) * 2 - 1)
        x = x.to(torch.bfloat16).float()
        scales[i:i + k] = _scale_of(x.abs().amax(-1))
        y = _codes(x, scales[i:i + k, :, None]).view(k, nblk * blk, d)
        codes[i:i + k] = y[:, :tokens]
    return codes, scales


def _cache(c, gen):
    """K, V and index key of the cache: codes [planes, rows, h, d] (a head's rows next to
    each other in memory) and scales [batch, blocks, h] or [pages, h]."""
    b, h, B, nblk = c["batch"], c["h"], c["block"], _blocks(c)
    planes, rows = (b * nblk + 3, B) if c["paged"] else (b, c["max_kv"])
    out = {}
    for name, heads, d in (("k", h, c["d"]), ("v", h, c["d"]), ("ki", 1, c["d_idx"])):
        codes, scales = _filled((planes * heads, rows, d), B, gen)
        codes = codes.view(planes, heads, rows, d).transpose(1, 2)
        scales = scales.view(planes, heads, -1).transpose(1, 2)
        scales = scales.squeeze(1) if c["paged"] else scales
        if name == "ki":
            codes, scales = codes.squeeze(2), scales.squeeze(-1)
        out[name], out[name + "_scale"] = codes, scales.contiguous()
    if c["paged"]:
        perm = torch.randperm(planes, device=DEV, generator=gen)[:b * nblk]
        out["table"] = perm.view(b, nblk).int()
    return out


def _rows(gen, *shape):
    return torch.randn(shape, device=DEV, generator=gen).to(torch.bfloat16)


def prepare(c, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    b, n, h, H, B, nblk = c["batch"], c["n"], c["h"], c["H"], c["block"], _blocks(c)
    s = {**c, "table": None, "nblk": nblk, **_cache(c, gen)}
    least = n if c["op"] == "append" else 0
    lens = torch.full((b,), c["max_kv"], device=DEV, dtype=torch.int32)
    if c["ragged"]:
        lens = torch.randint(least, c["max_kv"] + 1, (b,), device=DEV, generator=gen).int()
    s["lens"] = lens
    if c["op"] == "append":
        # new rows up to 4 times the size of the older ones: some blocks' scales grow
        grow = torch.exp2(torch.rand((b, n, h, 1), device=DEV, generator=gen) * 3 - 1)
        s["k_new"] = (_rows(gen, b, n, h, c["d"]) * grow).to(torch.bfloat16)
        s["v_new"] = _rows(gen, b, n, h, c["d"])
        s["ki_new"] = _rows(gen, b, n, c["d_idx"])
    elif c["op"] == "read":
        s["base"] = (c["max_kv"] - n) // 2
        s["k_out"] = torch.zeros((b, n, h, c["d"]), device=DEV, dtype=torch.bfloat16)
        s["v_out"] = torch.zeros_like(s["k_out"])
        s["ki_out"] = torch.zeros((b, n, c["d_idx"]), device=DEV, dtype=torch.bfloat16)
    elif c["op"] == "scores":
        s["q_idx"] = _rows(gen, b, n, h, c["d_idx"])
    else:
        s["q"] = _rows(gen, b, n, H, c["d"])
        # ids: a random choice among the blocks a query sees, ascending, -1 where there are fewer
        pos = lens[:, None] - n + torch.arange(n, device=DEV)
        seen = torch.arange(nblk, device=DEV) * B <= pos[..., None]  # [b, n, nblk]
        pick = torch.rand((b, n, h, nblk), device=DEV, generator=gen)
        pick = torch.where(seen[:, :, None], pick, -1.0)
        k = min(c["topk"], nblk)
        val, ids = pick.topk(k, dim=-1)
        ids = torch.where(val >= 0, ids, nblk).sort(-1).values
        ids = torch.where(ids < nblk, ids, -1)
        s["ids"] = torch.nn.functional.pad(ids, (0, c["topk"] - k), value=-1).int().contiguous()
    return s


# ------------------------------------------------------------- the plain forms
def _planes(s, blk, b):
    """Plane of the code tensors and of the scales, for block `blk` of sequence `b`."""
    return b if s["table"] is None else s["table"][b, blk].long()


def _append_one(s, codes, scales, new):
    """codes [planes, rows, h, d], scales [planes, (blocks,) h], new [b, n, h, d]."""
    B, n, cap = s["block"], s["n"], s["max_kv"]
    paged = s["table"] is not None
    raw = codes.view(torch.uint8)
    b = torch.arange(s["batch"], device=DEV)
    start = s["lens"].long() - n  # position of the first new row
    first = start // B
    pos = start[:, None] + torch.arange(n, device=DEV)
    blk = pos // B
    slot = blk - first[:, None]
    # scale that each touched block needs
    count = (n + B - 2) // B + 1
    new = new.float()
    need = torch.zeros((s["batch"], count, new.shape[2]), device=DEV)
    need = need.scatter_reduce(1, slot[..., None].expand(-1, -1, new.shape[2]),
                               new.abs().amax(-1), "amax")
    need = _scale_of(need)
    # the first block may hold older rows: its scale never shrinks
    first_plane = _planes(s, first, b)
    at = (first_plane,) if paged else (first_plane, first)
    old_scale = scales[at]
    held = (start % B > 0)[:, None]
    need[:, 0] = torch.where(held, torch.maximum(need[:, 0], old_scale), need[:, 0])
    # older rows of that block, rounded to its new scale
    off = torch.arange(B, device=DEV)
    row = (off.expand(s["batch"], B) if paged else (first[:, None] * B + off).clamp_max(cap - 1))
    tile = raw[first_plane[:, None], row]  # [b, B, h, d]
    value = tile.view(F8).float() * old_scale[:, None, :, None]
    again = _codes(value, need[:, :1, :, None]).view(torch.uint8)
    older = (off < (start % B)[:, None])[..., None, None]
    raw[first_plane[:, None], row] = torch.where(older, again, tile)
    # the new rows, and the scales of the touched blocks
    mine = need.gather(1, slot[..., None].expand(-1, -1, new.shape[2]))
    row = pos % B if paged else pos
    plane = _planes(s, blk, b[:, None]).expand_as(pos)
    raw[plane, row] = _codes(new, mine[..., None]).view(torch.uint8)
    touched = first[:, None] + torch.arange(count, device=DEV)
    live = touched * B < s["lens"][:, None]
    touched = torch.where(live, touched, first[:, None])
    value = torch.where(live[..., None], need, need[:, :1])
    plane = _planes(s, touched, b[:, None]).expand_as(touched)
    scales[(plane,) if paged else (plane, touched)] = value


def _append_plain(s):
    _append_one(s, s["k"], s["k_scale"], s["k_new"])
    _append_one(s, s["v"], s["v_scale"], s["v_new"])
    _append_one(s, s["ki"].unsqueeze(2), s["ki_scale"].unsqueeze(-1), s["ki_new"].unsqueeze(2))


def _read_one(s, codes, scales, out):
    n, B = s["n"], s["block"]
    b = torch.arange(s["batch"], device=DEV)[:, None]
    pos = s["base"] + torch.arange(n, device=DEV).expand(s["batch"], n)
    blk = pos // B
    plane = _planes(s, blk, b).expand_as(pos)
    paged = s["table"] is not None
    x = codes.view(torch.uint8)[plane, pos % B if paged else pos].view(F8).float()
    x = x * scales[(plane,) if paged else (plane, blk)][..., None]
    live = (pos < s["lens"][:, None])[..., None, None]
    out.copy_(torch.where(live, x.to(torch.bfloat16), out))


def _read_plain(s):
    _read_one(s, s["k"], s["k_scale"], s["k_out"])
    _read_one(s, s["v"], s["v_scale"], s["v_out"])
    _read_one(s, s["ki"].unsqueeze(2), s["ki_scale"].unsqueeze(-1), s["ki_out"].unsqueeze(2))


def _scores_plain(s):
    b, n, B, nblk = s["batch"], s["n"], s["block"], s["nblk"]
    raw, scale = s["ki"].view(torch.uint8), s["ki_scale"]
    if s["table"] is not None:
        raw = raw[s["table"].long()].view(b, nblk * B, -1)
        scale = scale[s["table"].long()]
    pad = nblk * B - raw.shape[1]
    raw = torch.nn.functional.pad(raw, (0, 0, 0, pad))
    key = raw.view(F8).float().view(b, nblk, B, -1) * scale[..., None, None]
    key = key.view(b, nblk * B, -1)
    q = s["q_idx"].float().view(b, n * s["h"], -1)
    dots = torch.matmul(q, key.transpose(1, 2)).view(b, n, s["h"], nblk * B)
    tok = torch.arange(nblk * B, device=DEV)
    lim = torch.minimum(s["lens"][:, None], s["lens"][:, None] - n + 1 + torch.arange(n, device=DEV))
    dots = torch.where(tok < lim[..., None, None], dots, -torch.inf)
    return dots.view(b, n, s["h"], nblk, B).amax(-1)


def _attn_plain(s):
    b, n, h, H, d, B = s["batch"], s["n"], s["h"], s["H"], s["d"], s["block"]
    ids = s["ids"].long()
    blk = ids.clamp_min(0)
    bi = torch.arange(b, device=DEV).view(b, 1, 1, 1)
    hi = torch.arange(h, device=DEV).view(1, 1, h, 1)
    plane = _planes(s, blk, bi).expand_as(blk)
    tok = blk[..., None] * B + torch.arange(B, device=DEV)  # [b, n, h, topk, B]
    lim = torch.minimum(s["lens"][:, None], s["lens"][:, None] - n + 1 + torch.arange(n, device=DEV))
    live = (ids[..., None] >= 0) & (tok < lim[:, :, None, None, None])
    row = tok % B if s["table"] is not None else tok.clamp_max(s["max_kv"] - 1)
    at = (plane, hi) if s["table"] is not None else (plane, blk, hi)
    where = (plane[..., None], row, hi[..., None])
    k = s["k"].view(torch.uint8)[where].view(F8).float()
    k *= s["k_scale"][at][..., None, None]
    v = s["v"].view(torch.uint8)[where].view(F8).float()
    v *= s["v_scale"][at][..., None, None]
    v.masked_fill_(~live[..., None], 0.0)
    k, v, live = k.flatten(3, 4), v.flatten(3, 4), live.flatten(3, 4)
    q = s["q"].float().view(b, n, h, H // h, d)
    x = torch.matmul(q, k.transpose(-1, -2)) * d ** -0.5
    x = torch.where(live[..., None, :], x, -torch.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top > -torch.inf, top, 0.0))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    lse = (top + torch.log(total)).view(b, n, H)
    return out.to(torch.bfloat16).view(b, n, H, d), lse


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "append":
        _append_plain(s)
        return _kept(s)
    if s["op"] == "read":
        _read_plain(s)
        return {"k": s["k_out"], "v": s["v_out"], "ki": s["ki_out"]}
    if s["op"] == "scores":
        return {"scores": _scores_plain(s)}
    out, lse = _attn_plain(s)
    return {"out": out, "lse": lse}


def _kept(s):
    """The cache after a write: the 8-bit values and their scales."""
    return {x: s[x] for x in ("k", "v", "ki", "k_scale", "v_scale", "ki_scale")}


def _run_own(s):
    from block_sparse_gqa_03_b200 import msa

    kw = dict(block=s["block"], seq_lens=s["lens"], block_table=s["table"], max_kv=s["max_kv"])
    cache = (s["k"], s["v"], s["ki"], s["k_scale"], s["v_scale"], s["ki_scale"])
    if s["op"] == "append":
        msa.msa_append_kv_q8(*cache, s["k_new"], s["v_new"], s["ki_new"], **kw)
        return _kept(s)
    if s["op"] == "read":
        k, v, ki = msa.msa_read_kv_q8(*cache, n=s["n"], token_base=s["base"], k_out=s["k_out"],
                                      v_out=s["v_out"], k_idx_out=s["ki_out"], **kw)
        return {"k": k, "v": v, "ki": ki}
    if s["op"] == "scores":
        return {"scores": msa.msa_block_scores_q8(s["q_idx"], s["ki"], s["ki_scale"], **kw)}
    out, lse = msa.msa_sparse_attn_q8(s["q"], s["k"], s["v"], s["k_scale"], s["v_scale"], s["ids"],
                                      return_lse=True, **kw)
    return {"out": out, "lse": lse}


# ------------------------------------------------------- the definitions in 64 bits
def _e4m3_values():
    """The 127 non-negative e4m3 values, by their code."""
    code = torch.arange(127, device=DEV, dtype=torch.float64)
    exp, frac = torch.floor(code / 8), code % 8
    return torch.where(exp > 0, (1 + frac / 8) * torch.exp2(exp - 7), frac / 8 * 2.0 ** -6)


def _nearest(x):
    """x rounded to the nearest e4m3 value, ties to the even code."""
    val = _e4m3_values()
    mid = (val[1:] + val[:-1]) / 2
    mag = x.abs().contiguous()
    lo = torch.searchsorted(mid, mag)
    hi = torch.searchsorted(mid, mag, right=True)
    return torch.sign(x) * val[torch.where(lo % 2 == 0, lo, hi)]


def _least_scale(amax):
    e = int(torch.ceil(torch.log2(torch.tensor(max(amax, 1e-300), dtype=torch.float64) / LARGEST)))
    while amax > LARGEST * 2.0 ** e:
        e += 1
    while amax <= LARGEST * 2.0 ** (e - 1) and e > -100:
        e -= 1
    return 2.0 ** max(e, -100)


def _exact_append(s):
    got = {}
    for name, new in (("k", s["k_new"]), ("v", s["v_new"]), ("ki", s["ki_new"].unsqueeze(2))):
        one = name == "ki"
        codes = s[name].unsqueeze(2) if one else s[name]
        scales = s[name + "_scale"].unsqueeze(-1) if one else s[name + "_scale"]
        val, scl, new = codes.double(), scales.double(), new.double()
        B, n = s["block"], s["n"]
        for b, length in enumerate(s["lens"].tolist()):
            pos = length - n
            while pos < length:
                blk, off = pos // B, pos % B
                stop = min(length, (blk + 1) * B)
                if s["table"] is None:
                    rows, sc = val[b, blk * B:stop], scl[b, blk]
                else:
                    page = int(s["table"][b, blk])
                    rows, sc = val[page, :stop - blk * B], scl[page]
                fresh = new[b, pos - (length - n):stop - (length - n)]
                most = fresh.abs().amax((0, 2)).tolist()
                need = torch.tensor([_least_scale(a) for a in most], device=DEV, dtype=torch.float64)
                kept = torch.maximum(need, sc) if off else need
                if off:
                    rows[:off] = _nearest(rows[:off] * (sc / kept)[:, None])
                rows[off:] = _nearest(fresh / kept[:, None])
                sc.copy_(kept)
                pos = stop
        got[name] = val.squeeze(2) if one else val
        got[name + "_scale"] = scl.squeeze(-1) if one else scl
    return got


def _whole(s, codes, scales, b):
    """Sequence b's values [tokens, h, d] in 64 bits, up to its capacity."""
    B, cap = s["block"], s["max_kv"]
    if s["table"] is None:
        x, sc = codes[b].double(), scales[b]
    else:
        page = s["table"][b].long()
        x = codes.view(torch.uint8)[page].view(F8).double().flatten(0, 1)
        sc = scales[page]
    return x[:cap] * sc.double().repeat_interleave(B, 0)[:x.shape[0]][:cap, :, None]


def _exact_read(s):
    got = {}
    for name in ("k", "v", "ki"):
        out = s[name + "_out"].double()
        codes, scales = s[name], s[name + "_scale"]
        if name == "ki":
            codes, scales = codes.unsqueeze(2), scales.unsqueeze(-1)
        for b, length in enumerate(s["lens"].tolist()):
            stop = min(length, s["base"] + s["n"])
            if stop > s["base"]:
                x = _whole(s, codes, scales, b)[s["base"]:stop]
                out[b, :stop - s["base"]] = x.squeeze(1) if name == "ki" else x
        got[name] = out
    return got


def _exact_scores(s):
    b, n, h, B, nblk = s["batch"], s["n"], s["h"], s["block"], s["nblk"]
    out = torch.full((b, n, h, nblk), -torch.inf, device=DEV, dtype=torch.float64)
    for i, length in enumerate(s["lens"].tolist()):
        key = _whole(s, s["ki"].unsqueeze(2), s["ki_scale"].unsqueeze(-1), i)[:length, 0]
        last = length - n + torch.arange(n, device=DEV)
        for g in range(h):
            x = s["q_idx"][i, :, g].double() @ key.T
            x[torch.arange(length, device=DEV) > last[:, None]] = -torch.inf
            x = torch.nn.functional.pad(x, (0, nblk * B - length), value=-torch.inf)
            out[i, :, g] = x.view(n, nblk, B).amax(-1)
    return {"scores": out}


def _exact_attn(s):
    b, n, h, H, d, B, nblk = (s[x] for x in ("batch", "n", "h", "H", "d", "block", "nblk"))
    G = H // h
    out = torch.zeros((b, n, H, d), device=DEV, dtype=torch.float64)
    lse = torch.full((b, n, H), -torch.inf, device=DEV, dtype=torch.float64)
    for i, length in enumerate(s["lens"].tolist()):
        if length == 0:
            continue
        k = _whole(s, s["k"], s["k_scale"], i)[:length]
        v = _whole(s, s["v"], s["v_scale"], i)[:length]
        last = length - n + torch.arange(n, device=DEV)
        for g in range(h):
            sel = torch.zeros((n, nblk + 1), device=DEV, dtype=torch.bool)
            ids = s["ids"][i, :, g].long()
            sel.scatter_(1, torch.where(ids < 0, nblk, ids), True)
            sel = sel[:, :nblk].repeat_interleave(B, 1)[:, :length]
            sel &= torch.arange(length, device=DEV) <= last[:, None]
            for j in range(G):
                x = s["q"][i, :, g * G + j].double() @ k[:, g].T / d ** 0.5
                x[~sel] = -torch.inf
                z = torch.logsumexp(x, -1)
                p = torch.exp(x - torch.where(z > -torch.inf, z, 0.0)[:, None])
                out[i, :, g * G + j] = p @ v[:, g]
                lse[i, :, g * G + j] = z
    return {"out": out, "lse": lse}


def exact(c, seed):
    s = prepare(c, seed)
    return {"append": _exact_append, "read": _exact_read, "scores": _exact_scores,
            "attn": _exact_attn}[c["op"]](s)
