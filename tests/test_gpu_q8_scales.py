"""The 8-bit cache's readers with scales that are no powers of two.

Tolerance of the scores: that of tests/q8_ref.py (2^-16 of the largest sum |q_i k_i| of the
block), and 2^-22 of it for the products with the scale (two roundings of 2^-24, and one of
the reference's scale, an fp32 number taken exactly).  A key that is rounded to bf16 before
the product is off by up to 2^-9 of it and does not pass."""

import pytest
import torch

import q8_ref
from block_sparse_gqa_03_b200 import msa

pytestmark = pytest.mark.gpu
DEV = "cuda"


def u8(t):
    return t.view(torch.uint8)


def free_cache(g, *, batch, max_kv, h, d, d_idx, block, paged):
    """Codes of normal values, scales anywhere in [2^-8, 2^-6)."""
    nblk = -(-max_kv // block)
    table = None
    if paged:
        table = torch.randperm(batch * nblk + 2, device=DEV, generator=g)[:batch * nblk]
        table = table.view(batch, nblk).int()
        c = msa.q8_cache(num_pages=batch * nblk + 2, h=h, d=d, d_idx=d_idx, block=block)
    else:
        c = msa.q8_cache(batch=batch, max_kv=max_kv, h=h, d=d, d_idx=d_idx, block=block)
    for codes in c[:3]:
        x = torch.randn(codes.shape, device=DEV, generator=g) * 100
        codes.copy_(x.clamp(-448, 448).to(torch.float8_e4m3fn))
    for s in c[3:]:
        s.copy_((1 + 3 * torch.rand(s.shape, device=DEV, generator=g)) * 2.0 ** -8)
    return c, table


def key_of(c, table, block, b, max_kv):
    return q8_ref.values(u8(c.k_idx).unsqueeze(2), c.k_idx_scale.unsqueeze(-1), block, b, max_kv,
                         table)[:, 0]


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("n,h,d_idx,block,max_kv,lens", [
    (1, 4, 128, 64, 700, [700, 65, 0]),
    (1, 9, 32, 16, 130, [130, 7]),
    (2, 3, 64, 64, 700, [700, 65, 1]),      # queries before the first token
    (150, 2, 128, 16, 500, [500, 333]),     # four scores to a store (32 blocks)
    (150, 2, 128, 16, 512, [512, 170]),
    (130, 3, 64, 32, 399, [399, 130]),
    (300, 2, 128, 128, 900, [900, 301]),
    (70, 5, 32, 32, 200, [200, 71]),        # the scan of 32-dim index keys
    (33, 1, 32, 128, 333, [333, 40]),
])
def test_scores(paged, n, h, d_idx, block, max_kv, lens):
    g = torch.Generator(device=DEV).manual_seed(n + h + d_idx)
    c, table = free_cache(g, batch=len(lens), max_kv=max_kv, h=1, d=64, d_idx=d_idx, block=block,
                          paged=paged)
    q = torch.randn((len(lens), n, h, d_idx), device=DEV, generator=g).to(torch.bfloat16)
    ws = msa.Workspace(DEV)
    kw = dict(block=block, seq_lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
              block_table=table, max_kv=max_kv, workspace=ws)
    got = msa.msa_block_scores_q8(q, c.k_idx, c.k_idx_scale, **kw)
    assert msa.msa_get_device_status(ws) == msa.MSA_OK
    for b, L in enumerate(lens):
        want, mag = q8_ref.scores(q[b].double(), key_of(c, table, block, b, max_kv), L, block)
        x, fin = got[b].double(), torch.isfinite(want)
        assert torch.equal(torch.isneginf(x), ~fin)
        assert bool(((x - want).abs()[fin] <= mag[fin] * (2.0 ** -16 + 2.0 ** -22)).all())


@pytest.mark.parametrize("d_idx", [32, 64, 128])
def test_a_prompt_and_a_step_rank_the_blocks_alike(d_idx):
    """Keys that differ from block to block by less than a bf16 rounding: the last query of a
    prompt selects the blocks that a step with the same query selects."""
    g = torch.Generator(device=DEV).manual_seed(d_idx)
    block, max_kv, h, topk = 16, 1024, 2, 5
    c, _ = free_cache(g, batch=1, max_kv=max_kv, h=1, d=64, d_idx=d_idx, block=block, paged=False)
    c.k_idx.copy_(c.k_idx[:, :block].repeat(1, max_kv // block, 1))
    order = torch.randperm(max_kv // block, device=DEV, generator=g)
    c.k_idx_scale.copy_((1 + order * 2.0 ** -12)[None])  # steps of 1/16 of a bf16 step
    q = torch.randn((1, 40, h, d_idx), device=DEV, generator=g).to(torch.bfloat16).abs()
    q[:, -1] = u8(c.k_idx)[:, 3:4].view(torch.float8_e4m3fn).float().to(torch.bfloat16)
    kw = dict(block=block, topk=topk, return_scores=True)
    many, s_many = msa.msa_index_select_q8(q, c.k_idx, c.k_idx_scale, **kw)
    one, s_one = msa.msa_index_select_q8(q[:, -1:].contiguous(), c.k_idx, c.k_idx_scale, **kw)
    best = order.argsort(descending=True)[:topk].sort().values.int()
    for g_ in range(h):
        assert torch.equal(one[0, 0, g_], best) and torch.equal(many[0, -1, g_], best)
    # the same sums of exact products up to their order
    assert bool(((s_many[0, -1] - s_one[0, 0]).abs() <= s_one[0, 0].abs() * 2.0 ** -14).all())


@pytest.mark.parametrize("paged", [False, True])
def test_scores_in_several_passes(paged):
    """Sequences of 1M tokens of capacity: the keys of four are widened at a time, six give two
    passes.  The same bits as one sequence at a time, and as the definition."""
    g = torch.Generator(device=DEV).manual_seed(5)
    batch, max_kv, block, h, di, n = 6, 1 << 20, 64, 2, 128, 3
    nblk = max_kv // block
    lens = [5000, 1, 70, max_kv if not paged else 9000, 0, 333]
    if paged:  # pages for the rows there are, and none behind them
        used = [-(-x // block) for x in lens]
        c, _ = free_cache(g, batch=1, max_kv=sum(used) * block, h=1, d=64, d_idx=di, block=block,
                          paged=True)
        table = torch.full((batch, nblk), -7, dtype=torch.int32, device=DEV)
        ids = torch.randperm(sum(used), device=DEV, generator=g).int()
        for b, k in enumerate(used):
            table[b, :k], ids = ids[:k], ids[k:]
        key, scale = c.k_idx, c.k_idx_scale
    else:
        table = None
        key = torch.randint(0, 120, (batch, max_kv, di), device=DEV, generator=g, dtype=torch.uint8)
        scale = torch.rand((batch, nblk), device=DEV, generator=g) + 0.5
    q = torch.randn((batch, n, h, di), device=DEV, generator=g).to(torch.bfloat16)
    ws = msa.Workspace(DEV)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    kw = dict(block=block, max_kv=max_kv, workspace=ws, topk=4, return_scores=True)
    ids, got = msa.msa_index_select_q8(q, key, scale, seq_lens=sl, block_table=table, **kw)
    assert msa.msa_get_device_status(ws) == msa.MSA_OK
    assert ws.buf.numel() < (1 << 30) + (1 << 24)
    for b, L in enumerate(lens):
        part = slice(b, b + 1)
        one_ids, one = msa.msa_index_select_q8(
            q[part], key if paged else key[part], scale if paged else scale[part],
            seq_lens=sl[part], block_table=None if table is None else table[part], **kw)
        assert torch.equal(one, got[part]) and torch.equal(one_ids, ids[part])
        m = min(L, 5000)
        if paged:
            page = table[b, :-(-L // block)].long()
            val = q8_ref.decode(u8(key)[page]) * scale[page].double()[:, None, None]
            val = val.flatten(0, 1)[:m]
        else:
            val = q8_ref.decode(key[b, :m]) * scale[b].double().repeat_interleave(block)[:m, None]
        if m == L and L > 0:
            want, mag = q8_ref.scores(q[b].double(), val, L, block)
            x, fin = got[b, :, :, :want.shape[-1]].double(), torch.isfinite(want)
            assert torch.equal(torch.isneginf(x), ~fin)
            assert bool(((x - want).abs()[fin] <= mag[fin] * (2.0 ** -16 + 2.0 ** -22)).all())
        assert bool(torch.isneginf(got[b, :, :, -(-L // block):]).all())
    assert msa.msa_get_device_status(ws) == msa.MSA_OK
