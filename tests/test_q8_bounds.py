"""The bounds of q8_bounds.py on the CPU: a merge of f16 partial outputs keeps them, one of
bf16 partial outputs does not."""

import pytest
import torch

import q8_bounds
import q8_ref


def merged(q, k, v, vs, ids, block, scale, part):
    """The by-block method of one sequence in 64 bits, its partial outputs rounded to
    ``part`` in units of the V scale, the result to bf16."""
    n, H, d = q.shape
    G = H // k.shape[1]
    out = torch.zeros((n, H, d), dtype=torch.float64)
    for t in range(n):
        for hq in range(H):
            g = hq // G
            acc, den, top = 0.0, 0.0, -torch.inf
            parts = []
            for beta in ids[t, g].tolist():
                j = slice(beta * block, (beta + 1) * block)
                x = (k[j, g] @ q[t, hq]) * scale
                m = x.max()
                p = torch.exp(x - m)
                o = (p @ (v[j, g] / vs[j, g, None])) / p.sum()
                parts.append((o.to(part).double() * vs[j.start, g], m + torch.log(p.sum())))
                top = max(top, float(parts[-1][1]))
            for o, z in parts:
                w = torch.exp(z - top)
                acc, den = acc + w * o, den + w
            out[t, hq] = acc / den
    return out.to(torch.bfloat16).double()


@pytest.mark.parametrize("part", [torch.float16, torch.bfloat16])
def test_bound_tells_f16_from_bf16_partial_outputs(part):
    """Two blocks a query whose values have opposite signs: the output is the small difference
    of two partial outputs."""
    g = torch.Generator().manual_seed(1)
    n, H, h, d, block = 40, 4, 2, 64, 64
    L = 4 * block
    codes = (torch.randn((3, L, h, d), generator=g) * 100).clamp(-448, 448)
    codes = codes.to(torch.float8_e4m3fn).double()
    k = codes[0] * 2.0 ** -9
    vs = torch.full((L, h), 2.0 ** -7)
    sign = torch.where(torch.arange(L) // block % 2 == 0, 1.0, -1.0)[:, None, None]
    v = codes[1].abs() * sign * 2.0 ** -7
    q = torch.randn((n, H, d), generator=g).to(torch.bfloat16).double()
    ids = torch.tensor([[0, 1], [2, 3]])[torch.randint(0, 2, (n, h), generator=g)]
    scale = d ** -0.5
    o, z, more = q8_bounds.reference(q, k, v, vs, ids, L, block, scale, causal=False)
    got = merged(q, k, v, vs, ids, block, scale, part)
    bound, _ = q8_bounds.bounds(o, z, *more[:5], by_block=True, U=more[5])
    assert bool(((got - o).abs() <= bound).all()) == (part == torch.float16)
    # without partial outputs the bound is tighter still, and with the allowance for bf16 ones
    # neither mistake would be seen
    loose = q8_ref.out_bound(o, more[0], more[1], more[2], more[3], True)
    assert bool(((got - o).abs() <= loose).all())
