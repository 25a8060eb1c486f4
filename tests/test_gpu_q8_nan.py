"""NaN in the 8-bit attention's inputs: a row that sees one is NaN, on every path, and one
that does not see it keeps its bits."""

import pytest
import torch

import q8_bounds
from block_sparse_gqa_03_b200 import msa
from test_gpu_q8_paths import filled, gen, pick, rows, u8

pytestmark = pytest.mark.gpu
DEV = "cuda"

CASES = [
    # path, n, H, h, d, block, topk, max_kv, lens
    ("streamed", 1, 16, 2, 128, 64, 60, 9000, [9000, 5000, 0]),   # split rows
    ("streamed", 1, 16, 1, 64, 16, 90, 2000, [2000, 1300]),
    ("streamed", 70, 8, 2, 128, 64, 4, 400, [300, 70]),
    ("by row", 160, 8, 2, 128, 64, 4, 400, [300, 150]),           # queries before the first token
    ("by row", 700, 12, 1, 64, 32, 40, 1700, [1700]),
    ("by block", 1100, 8, 2, 128, 64, 4, 1200, [1150, 1090]),
    ("by block", 1100, 32, 4, 64, 64, 5, 1100, [1100]),
    ("by block", 1100, 32, 4, 128, 128, 3, 1100, [1100]),
    ("by block", 2100, 26, 2, 64, 128, 16, 2100, [2100]),
    ("by block", 2100, 4, 2, 64, 64, 33, 2100, [2100]),
]


def problem(way, n, H, h, d, block, topk, max_kv, lens, paged):
    assert q8_bounds.path(len(lens), n, H, h, d, block, topk, max_kv) == way
    g = gen(n + H + d + topk)
    c, table = filled(g, batch=len(lens), max_kv=max_kv, h=h, d=d, block=block, paged=paged,
                      scales="free")
    q = rows(g, len(lens), n, H, d)
    ids = pick(g, lens, n, h, -(-max_kv // block), block, topk)
    kw = dict(block=block, block_table=table, max_kv=max_kv, return_lse=True,
              seq_lens=torch.tensor(lens, dtype=torch.int32, device=DEV))

    def run():
        return msa.msa_sparse_attn_q8(q, c.k, c.v, c.k_scale, c.v_scale, ids, **kw)

    return g, c, table, q, ids, run


def visible(ids, b, L, n, h, block, max_kv):
    """bool [n, h, max_kv]: the tokens that a (query, group) of sequence b selects and sees."""
    nblk = -(-max_kv // block)
    sel = torch.zeros((n, h, nblk + 1), dtype=torch.bool, device=DEV)
    sel.scatter_(2, torch.where(ids[b] < 0, nblk, ids[b]).long(), True)
    sel = sel[..., :nblk].repeat_interleave(block, 2)[..., :max_kv]
    j = torch.arange(max_kv, device=DEV)
    pos = L - n + torch.arange(n, device=DEV)
    return sel & (j < L) & (j <= pos[:, None])[:, None]


def put(codes, table, block, b, j, g, dims, value=0x7f):
    """Sets the code of token j of sequence b and head g."""
    raw = u8(codes)
    if table is None:
        raw[b, j, g, dims] = value
    else:
        raw[int(table[b, j // block]), j % block, g, dims] = value


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_a_visible_nan_key_or_query_makes_the_row_nan(case, paged):
    way, n, H, h, d, block, topk, max_kv, lens = case
    g, c, table, q, ids, run = problem(*case, paged)
    clean = run()
    bad = torch.zeros((len(lens), max_kv, h), dtype=torch.bool, device=DEV)
    for b, L in enumerate(lens):
        spots = torch.randint(0, max(L, 1), (3,), device=DEV, generator=g).tolist()
        spots += [max(L - 1, 0), max(L - n, 0)]
        # single codes, the last token among them, and one whole block of head 0
        for i, j in enumerate(spots):
            put(c.k, table, block, b, j, i % h, (7 * i) % d)
            bad[b, j, i % h] = True
        beta = L // block // 2
        for j in range(beta * block, min((beta + 1) * block, max_kv)):
            put(c.k, table, block, b, j, 0, slice(None))
            bad[b, j, 0] = True
    for t, hq in ((0, 0), (n // 2, H - 1), (n - 1, H // 2)):
        q[:, t, hq, 5] = torch.nan
    out, lse = run()
    G = H // h
    for b, L in enumerate(lens):
        see = visible(ids, b, L, n, h, block, max_kv)
        hit = (see & bad[b].T).any(-1).repeat_interleave(G, 1)
        hit |= torch.isnan(q[b]).any(-1) & see.any(-1).repeat_interleave(G, 1)
        assert bool(torch.isnan(out[b][hit]).all()) and bool(torch.isnan(lse[b][hit]).all())
        assert torch.equal(out[b][~hit], clean[0][b][~hit])
        assert torch.equal(lse[b][~hit], clean[1][b][~hit])
        assert bool(hit.any()) == (L > 0)
        if n > 1 and 4 * topk * block < max_kv:
            assert not bool(hit.all())


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_a_nan_value_reaches_the_rows_that_see_it_and_no_others(case, paged):
    """Values behind a query's position are masked: one that is NaN must not reach it, in a
    block that later queries see or in any other."""
    way, n, H, h, d, block, topk, max_kv, lens = case
    g, c, table, q, ids, run = problem(*case, paged)
    # zeros where NaN will be: the other rows' bits are those of this cache
    bad = torch.zeros((len(lens), max_kv, h, d), dtype=torch.bool, device=DEV)
    spots = []
    for b, L in enumerate(lens):
        at = torch.randint(0, max(L, 1), (4,), device=DEV, generator=g).tolist()
        at += [max(L - 1, 0), max(L - n, 0), max(L - 1 - n // 2, 0), 0]
        for i, j in enumerate(at):
            dims = torch.randint(0, d, (3,), device=DEV, generator=g)
            dims[0] = (d - 1, 0, d // 2)[i % 3]
            spots.append((b, j, i % h, dims, (0x7f, 0xff)[i % 2]))
            bad[b, j, i % h, dims] = j < L
    for b, j, head, dims, _ in spots:
        put(c.v, table, block, b, j, head, dims, 0)
    clean = run()
    assert bool(torch.isfinite(clean[0]).all())
    for b, j, head, dims, code in spots:
        put(c.v, table, block, b, j, head, dims, code)
    out, lse = run()
    G = H // h
    assert torch.equal(lse, clean[1])
    for b, L in enumerate(lens):
        see = visible(ids, b, L, n, h, block, max_kv)
        hit = torch.einsum("nhj,jhd->nhd", see.float(), bad[b].float()).repeat_interleave(G, 1) > 0
        assert bool(torch.isnan(out[b][hit]).all())
        assert torch.equal(out[b][~hit], clean[0][b][~hit])
        assert L == 0 or n == 1 or (bool(hit.any()) and not bool(hit.all()))
    again = run()
    assert torch.equal(u8(again[0]), u8(out))
    for b, j, head, dims, _ in spots:  # and nothing of it stays in the workspace
        put(c.v, table, block, b, j, head, dims, 0)
    assert torch.equal(run()[0], clean[0])
