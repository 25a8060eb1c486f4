"""Tolerances of the 8-bit attention by the path that a shape takes, to q8_ref.py's
derivation, and which path that is.

Streamed and by row: probabilities f16, everything behind them fp32: q8_ref.out_bound without
partial outputs.  Free scales (no powers of two) add the roundings of scale * s^K and of its
product with the score (2^-24 each, twice: 2^-22 of sum |q k| in dx) and of the product with
s^V (2^-24 A).

By block: a block's output is a mean of codes rounded to f16, 2^-11 of it, or 2^-25 in units
of s^V below f16's smallest normal number, weighted by the block's share w of the
probabilities: 2^-11 A + 2^-25 U with U = sum w s^V.  The weights e^(lse - M) come from
exponentials whose argument, of at most 2^8, is off by 2^-24 of it, and of the two ends by
log2 and the product with ln 2 (2^-16 together), and are off by 2 + 1.2 |argument| units of
2^-23 themselves (2^-18 for arguments above -25, below which a weight does not count):
2^-15 A."""

import torch

import q8_ref
from block_sparse_gqa_03_b200 import msa


def path(batch, n, H, h, d, block, topk, max_kv):
    """'streamed', 'by row' or 'by block' on the current device."""
    p = msa.make_params(batch=batch, n_q=n, max_kv=max_kv, H=H, h=h, d=d, d_idx=32, block=block,
                        topk=topk)
    launches = msa.msa_launch_count(p, msa.MSA_OP_SPARSE_ATTN_Q8)
    if launches > 1:
        return "by block"
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return "streamed" if batch * n * h < 4 * sms else "by row"


def bounds(out, lse, A, dx, total, N, mag, by_block, U):
    """Bounds of out [n, H, d] and lse [n, H]; ``mag``: the largest scale * sum |q k| of a
    row; ``U``: sum of w s^V [n, H, d]."""
    dx = dx + mag * 2.0 ** -22
    b = q8_ref.out_bound(out, A, dx, total, N, False) + A * 2.0 ** -24
    z = q8_ref.lse_bound(lse, dx)
    if by_block:
        b = b + A * (2.0 ** -11 + 2.0 ** -15) * 1.01 + U * 2.0 ** -25
        z = z + 2.0 ** -15  # __logf of the merged sum, and the weights' errors in it
    return b, z


def reference(q, k, v, vs, ids, L, block, scale, causal=True):
    """q8_ref.attention of one sequence, with ``vs`` [max_kv, h] the V scale of every token:
    (out, lse, arguments of bounds())."""
    o, z, A, dx, total, N = q8_ref.attention(q, k, v, ids, L, block, scale, causal)
    wide = vs.double()[..., None].expand(vs.shape + v.shape[-1:])
    U = q8_ref.attention(q, k, wide, ids, L, block, scale, causal)[2]
    return o, z, (A, dx, total, N, dx * 2.0 ** 16, U)
