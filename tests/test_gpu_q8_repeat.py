"""The streamed 8-bit attention gives the same bits at every run, whichever CTA of a split row
comes last and merges it."""

import pytest
import torch

from block_sparse_gqa_03_b200 import msa
from test_gpu_q8_paths import filled, gen, pick, rows

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("H,h,d,block,topk,max_kv,lens", [
    # rows of seven segments and more; with the second sequence shorter than its list, the CTA
    # that ends the first row has little behind it and often comes last
    (16, 1, 64, 16, 90, 2000, [2000, 1300]),
    (16, 1, 128, 16, 90, 2000, [2000, 1300]),
    (8, 1, 64, 16, 200, 6000, [6000, 700, 6000, 20]),
    (8, 1, 128, 32, 200, 9000, [9000, 100, 9000, 100]),
    (6, 2, 64, 64, 300, 30000, [30000, 5000, 30000]),
    (8, 1, 128, 64, 1000, 64000, [64000]),     # one row over many CTAs
    (48, 3, 128, 128, 400, 60000, [60000]),
    (16, 1, 64, 64, 500, 40000, [40000, 3000]),
])
def test_split_rows_repeat_their_bits(H, h, d, block, topk, max_kv, lens):
    g, batch = gen(topk), len(lens)
    nblk = -(-max_kv // block)
    c, table = filled(g, batch=batch, max_kv=max_kv, h=h, d=d, block=block, paged=True,
                      scales="free")
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    a = torch.randn((1024, 1024), device=DEV).to(torch.bfloat16)
    side.wait_stream(torch.cuda.current_stream())
    for draw in range(60):  # an order shows where its roundings differ: in few heads of a draw
        q, ids = rows(g, batch, 1, H, d), pick(g, lens, 1, h, nblk, block, topk)

        def run():
            return msa.msa_sparse_attn_q8(q, c.k, c.v, c.k_scale, c.v_scale, ids, block=block,
                                          seq_lens=sl, block_table=table, max_kv=max_kv,
                                          return_lse=True)

        got = [run() for _ in range(30)]
        with torch.cuda.stream(side):  # beside other work, which changes the order further
            for _ in range(10):
                torch.mm(a, a)
        got += [run() for _ in range(10)]
        for out, lse in got[1:]:
            assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1]), draw
    torch.cuda.synchronize()


@pytest.mark.parametrize("n,H,h,d,block,topk,max_kv,lens", [
    (700, 12, 2, 64, 32, 6, 900, [900, 800]),        # by row
    (1100, 32, 4, 64, 64, 5, 1100, [1100]),          # by block, whose lists are filled by atomics
    (1300, 10, 2, 128, 128, 6, 1400, [1400, 1301]),
])
def test_prompts_repeat_their_bits(n, H, h, d, block, topk, max_kv, lens):
    g, batch = gen(n), len(lens)
    c, _ = filled(g, batch=batch, max_kv=max_kv, h=h, d=d, block=block, paged=False, scales="free")
    q, ids = rows(g, batch, n, H, d), pick(g, lens, n, h, -(-max_kv // block), block, topk)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    want = None
    for _ in range(60):
        got = msa.msa_sparse_attn_q8(q, c.k, c.v, c.k_scale, c.v_scale, ids, block=block,
                                     seq_lens=sl, return_lse=True)
        want = want or got
        assert all(torch.equal(a, b) for a, b in zip(got, want))
