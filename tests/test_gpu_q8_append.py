"""The 8-bit cache's write where its inputs are out of range."""

import pytest
import torch

from block_sparse_gqa_03_b200 import msa

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("n", [1, 5, 40])
def test_a_length_out_of_range_leaves_its_sequence_as_it_is(paged, n):
    """A step past the end of the cache (the last rows and the scales of their blocks must
    survive it), lengths far beyond it and below zero; the other sequences are written."""
    g = torch.Generator(device=DEV).manual_seed(n)
    batch, max_kv, h, d, di, block = 5, 50, 2, 64, 32, 16
    nblk = -(-max_kv // block)
    table = None
    if paged:
        table = torch.randperm(batch * nblk, device=DEV, generator=g).view(batch, nblk).int()
        c = msa.q8_cache(num_pages=batch * nblk, h=h, d=d, d_idx=di, block=block)
    else:
        c = msa.q8_cache(batch=batch, max_kv=max_kv, h=h, d=d, d_idx=di, block=block)

    def new(rows, f):
        return [(torch.randn((batch, rows) + s, device=DEV, generator=g) * f).to(torch.bfloat16)
                for s in ((h, d), (h, d), (di,))]

    ws = msa.Workspace(DEV)
    kw = dict(block=block, block_table=table, max_kv=max_kv, workspace=ws)
    msa.msa_append_kv_q8(*c, *new(max_kv, 1.0), **kw)
    assert msa.msa_get_device_status(ws) == msa.MSA_OK
    before = [t.clone() for t in c]
    # rows 64 times the older ones: a block that took one would get a larger scale
    lens = torch.tensor([max_kv + 1, max_kv, -1, 2**31 - 1, max_kv + n], dtype=torch.int32, device=DEV)
    msa.msa_append_kv_q8(*c, *new(n, 64.0), seq_lens=lens, **kw)
    assert msa.msa_get_device_status(ws) == msa.MSA_ERR_DEVICE_ASSERT
    for old, now in zip(before, c):
        where = (lambda b: b) if table is None else (lambda b: table[b].long())
        for b in (0, 2, 3, 4):
            assert torch.equal(old[where(b)].view(torch.uint8), now[where(b)].view(torch.uint8)), b
        assert not torch.equal(old[where(1)].view(torch.uint8), now[where(1)].view(torch.uint8))
