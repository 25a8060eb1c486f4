"""The 8-bit cache's operations in 64 bits, by their definitions (torch, any device).

Nothing here uses the library or torch's float8 conversions: codes are looked up in the
table of e4m3 values.

Tolerances.  A rounding is off by at most half a step: 2^-8 of the value for bf16, 2^-11
for f16, 2^-24 for fp32.
  scores  the products q_i c_i are exact in fp32; their sum over d_idx <= 128 terms is off
          by at most 128 * 2^-23 of sum |q_i k_i| (2^-23: a sum that truncates), 2^-16 of it.
  out     with x_j the scores, each off by at most dx = 2^-16 * scale * sum |q k| (as
          above), p_j is off by a factor e^dx, so out by 2 dx A with A = sum p_j |v_j| /
          sum p_j.  The probabilities' f16 rounding gives 2^-11 A and, below 2^-14 where
          the f16 step is fixed, 2^-25 sum |v_j| (a row's largest probability is 1, so the
          denominator is at least 1).  fp32 sums over N keys: N 2^-23 A.  exp2 and its
          argument (at most 2^8 in magnitude, off by 2^-24 of it): 2^-15 A.  The output's
          rounding: 2^-8 |out|.  Where partial outputs are rounded to bf16: 2^-8 A more.
  lse     dx, and 2^-15 for exp2 and log2 and their sums, and 2^-22 of the value.
"""

import torch

LARGEST = 448.0


def e4m3_values(device="cpu"):
    """The 127 non-negative values by their code, in 64 bits."""
    v = [(1 + c % 8 / 8) * 2.0 ** (c // 8 - 7) if c >= 8 else c * 2.0 ** -9 for c in range(127)]
    return torch.tensor(v, dtype=torch.float64, device=device)


def encode(x):
    """Codes (uint8) of float64 values: nearest, ties to even, saturating, NaN -> 0x7f."""
    val = e4m3_values(x.device)
    mid = (val[1:] + val[:-1]) / 2
    mag = torch.nan_to_num(x.abs(), nan=0.0, posinf=LARGEST).clamp_max(LARGEST).contiguous()
    lo, hi = torch.searchsorted(mid, mag), torch.searchsorted(mid, mag, right=True)
    code = torch.where(lo % 2 == 0, lo, hi)
    code = torch.where(torch.isnan(x), 127, code)
    neg = torch.signbit(x) & ~torch.isnan(x)
    return (code + 128 * neg).to(torch.uint8)


def decode(codes):
    """float64 values of codes (uint8)."""
    val = torch.cat([e4m3_values(codes.device),
                     torch.full((1,), torch.nan, dtype=torch.float64, device=codes.device)])
    c = codes.long()
    return torch.where(c >= 128, -val[c % 128], val[c % 128])


def scale_for(amax):
    """Smallest power of two s >= 2^-100 with amax <= 448 s (a float)."""
    s = 2.0 ** -100
    while amax > LARGEST * s:
        s *= 2
    return s


def append_one(codes, scales, new, lens, block, table=None):
    """codes uint8 [planes, rows, h, d], scales float64 [planes, (nblk,) h], new float64
    [b, n, h, d]; changed in place."""
    n = new.shape[1]
    for b, L in enumerate(lens):
        pos = max(L - n, 0)
        while pos < L:
            beta, off = pos // block, pos % block
            stop = min(L, (beta + 1) * block)
            if table is None:
                rows, sc = codes[b, beta * block:stop], scales[b, beta]
            else:
                page = int(table[b, beta])
                rows, sc = codes[page, :stop - beta * block], scales[page]
            fresh = new[b, pos - (L - n):stop - (L - n)]
            for g in range(new.shape[2]):
                x = fresh[:, g]
                fin = x[torch.isfinite(x)].abs()
                s = scale_for(float(fin.max()) if fin.numel() else 0.0)
                if off:
                    s = max(s, float(sc[g]))
                    rows[:off, g] = encode(decode(rows[:off, g]) * (float(sc[g]) / s))
                rows[off:, g] = encode(x / s)
                sc[g] = s
            pos = stop


def values(codes, scales, block, b, max_kv, table=None):
    """float64 [max_kv, h, d] of sequence b; codes [planes, rows, h, d]."""
    if table is None:
        x, sc = decode(codes[b]), scales[b]
    else:
        page = table[b].long()
        x, sc = decode(codes[page]).flatten(0, 1), scales[page]
    sc = sc.double().repeat_interleave(block, 0)
    return x[:max_kv] * sc[:max_kv, :, None]


def scores(q_idx, key, L, block, causal=True):
    """Block scores of one sequence: q_idx [n, h, di], key [max_kv, di] float64; and, per
    block, the largest sum |q_i k_i| of its visible tokens."""
    n, h, _ = q_idx.shape
    nblk = -(-key.shape[0] // block)
    pos = L - n + torch.arange(n, device=key.device)
    j = torch.arange(nblk * block, device=key.device)
    see = (j < L) & ((j <= pos[:, None]) if causal else torch.ones((n, 1), dtype=torch.bool,
                                                                   device=key.device))
    key = torch.nn.functional.pad(torch.where((j[:key.shape[0]] < L)[:, None], key, 0.0),
                                  (0, 0, 0, nblk * block - key.shape[0]))
    x = torch.einsum("nhd,jd->nhj", q_idx, key)
    mag = torch.einsum("nhd,jd->nhj", q_idx.abs(), key.abs())
    x = torch.where(see[:, None], x, -torch.inf).view(n, h, nblk, block).amax(-1)
    mag = torch.where(see[:, None], mag, 0.0).view(n, h, nblk, block).amax(-1)
    return x, mag


def attention(q, k, v, ids, L, block, scale, causal=True):
    """One sequence: q [n, H, d], k, v [max_kv, h, d], ids [n, h, topk]; out [n, H, d], lse
    [n, H], and what the tolerances above need: A [n, H, d], dx [n, H], sum |v| [n, H, d]
    and N [n, H]."""
    n, H, d = q.shape
    h, cap = k.shape[1], k.shape[0]
    G = H // h
    nblk = -(-cap // block)
    dev = q.device
    j = torch.arange(cap, device=dev)
    live = j < L
    k, v = torch.where(live[:, None, None], k, 0.0), torch.where(live[:, None, None], v, 0.0)
    pos = L - n + torch.arange(n, device=dev)
    see = live & ((j <= pos[:, None]) if causal else live.expand(n, cap))
    sel = torch.zeros((n, h, nblk + 1), dtype=torch.bool, device=dev)
    sel.scatter_(2, torch.where((ids < 0) | (ids >= nblk), nblk, ids).long(), True)
    sel = sel[..., :nblk].repeat_interleave(block, 2)[..., :cap] & see[:, None]
    sel = sel.repeat_interleave(G, 1)
    kk, vv = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    x = torch.einsum("nhd,jhd->nhj", q, kk) * scale
    mag = torch.einsum("nhd,jhd->nhj", q.abs(), kk.abs()) * abs(scale)
    x = torch.where(sel, x, -torch.inf)
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - torch.where(lse > -torch.inf, lse, 0.0)[..., None])
    dx = torch.where(sel, mag, 0.0).amax(-1) * 2.0 ** -16
    out = torch.einsum("nhj,jhd->nhd", p, vv)
    A = torch.einsum("nhj,jhd->nhd", p, vv.abs())
    total = torch.einsum("nhj,jhd->nhd", sel.double(), vv.abs())
    return out, lse, A, dx, total, sel.sum(-1)


def out_bound(out, A, dx, total, N, partials):
    c = 2 * dx + 2.0 ** -11 + N * 2.0 ** -23 + 2.0 ** -15 + (2.0 ** -8 if partials else 0.0)
    return out.abs() * 2.0 ** -8 + c[..., None] * A * 1.01 + total * 2.0 ** -25


def lse_bound(lse, dx):
    return dx + 2.0 ** -15 + torch.nan_to_num(lse.abs(), posinf=0.0) * 2.0 ** -22
