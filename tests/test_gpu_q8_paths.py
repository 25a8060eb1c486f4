"""8-bit attention on each of its three paths (streamed, one CTA per row, by block), the path
asserted, against the definition in 64 bits within the bounds of tests/q8_bounds.py."""

import pytest
import torch

import q8_bounds
import q8_ref
from block_sparse_gqa_03_b200 import msa

pytestmark = pytest.mark.gpu
DEV = "cuda"
F8 = torch.float8_e4m3fn


def u8(t):
    return t.view(torch.uint8)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def rows(g, *shape):
    return torch.randn(shape, device=DEV, generator=g).to(torch.bfloat16)


def filled(g, *, batch, max_kv, h, d, block, paged, scales):
    """Codes of normal values.  Scales: 'free', anywhere in [2^-8, 2^-6); 'apart', powers of two
    with V's from 2^-40 to 2^20 over a sequence's blocks."""
    nblk = -(-max_kv // block)
    table = None
    if paged:
        table = torch.randperm(batch * nblk + 2, device=DEV, generator=g)[:batch * nblk]
        table = table.view(batch, nblk).int()
        c = msa.q8_cache(num_pages=batch * nblk + 2, h=h, d=d, d_idx=32, block=block)
    else:
        c = msa.q8_cache(batch=batch, max_kv=max_kv, h=h, d=d, d_idx=32, block=block)
    for codes in (c.k, c.v):
        x = torch.randn(codes.shape, device=DEV, generator=g) * 100
        codes.copy_(x.clamp(-448, 448).to(F8))
    for s in (c.k_scale, c.v_scale):
        if scales == "free":
            s.copy_((1 + 3 * torch.rand(s.shape, device=DEV, generator=g)) * 2.0 ** -8)
        else:
            lo, hi = (-8, -5) if s is c.k_scale else (-40, 20)
            s.copy_(torch.exp2(torch.randint(lo, hi + 1, s.shape, device=DEV, generator=g).float()))
    return c, table


def pick(g, lens, n, h, nblk, block, topk):
    """Random distinct visible blocks in random order, -1 behind them."""
    key = torch.rand((len(lens), n, h, nblk), device=DEV, generator=g)
    for b, L in enumerate(lens):
        pos = L - n + torch.arange(n, device=DEV)
        seen = torch.arange(nblk, device=DEV) * block <= pos[:, None]
        key[b] = torch.where(seen[:, None], key[b], -1.0)
    k = min(topk, nblk)
    val, ids = key.topk(k, -1)
    ids = torch.where(val >= 0, ids, -1).int()
    return torch.nn.functional.pad(ids, (0, topk - k), value=-1).contiguous()


def check(c, table, q, ids, lens, block, max_kv, out, lse, by_block):
    scale = q.shape[-1] ** -0.5
    for b, L in enumerate(lens):
        k = q8_ref.values(u8(c.k), c.k_scale, block, b, max_kv, table)
        v = q8_ref.values(u8(c.v), c.v_scale, block, b, max_kv, table)
        vs = c.v_scale[b] if table is None else c.v_scale[table[b].long()]
        vs = vs.repeat_interleave(block, 0)[:max_kv]
        for t in range(0, q.shape[1], 500):  # a part of the queries at a time
            part = slice(t, t + 500)
            last = L - q.shape[1] + min(t + 500, q.shape[1])
            # the part's queries are the last ones of a sequence of `last` tokens
            qq, ii = q[b, part].double(), ids[b, part]
            o, z, more = q8_bounds.reference(qq, k, v, vs, ii, last, block, scale)
            ob, zb = q8_bounds.bounds(o, z, *more[:5], by_block=by_block, U=more[5])
            x, y = out[b, part].double(), lse[b, part].double()
            assert torch.equal(torch.isneginf(y), torch.isneginf(z))
            err = (x - o).abs()
            assert bool((err <= ob).all()), "sequence %d: error %g, bound there %g" % (
                b, float((err - ob).max()), float(ob.flatten()[(err - ob).argmax()]))
            fin = torch.isfinite(z)
            assert bool(((y - z).abs()[fin] <= zb[fin]).all())


CASES = [
    # path, n, H, h, d, block, topk, max_kv, lens
    ("streamed", 1, 16, 2, 128, 64, 6, 900, [900, 65, 1, 0]),
    ("streamed", 1, 12, 1, 64, 16, 9, 300, [300, 17]),
    ("streamed", 130, 8, 2, 128, 64, 4, 1200, [256, 250]),
    ("by row", 1, 16, 8, 128, 64, 5, 700, [700 - 8 * i for i in range(80)]),       # two warps
    ("by row", 1, 16, 8, 64, 128, 9, 1300, [1300 - 16 * i for i in range(76)]),    # four warps
    ("by row", 160, 8, 2, 128, 64, 4, 1200, [256, 250]),
    ("by row", 300, 22, 2, 64, 128, 2, 400, [400, 333]),
    ("by row", 700, 16, 2, 64, 32, 3, 700, [700]),
    ("by row", 800, 4, 1, 128, 128, 9, 1300, [1300]),        # 236 MB of blocks
    ("by block", 1300, 4, 1, 128, 128, 9, 1300, [1300]),     # and 383
    ("by block", 1100, 8, 2, 128, 64, 4, 1200, [1150, 1100]),
    ("by block", 1100, 32, 4, 64, 64, 5, 1100, [1100]),      # groups of 8 heads of 64 dims
    ("by block", 1100, 32, 4, 64, 128, 4, 1100, [1100]),
    ("by block", 1100, 32, 4, 128, 128, 3, 1100, [1100]),
    ("by block", 600, 32, 4, 128, 64, 5, 620, [600, 601]),   # and of 128 dims
    ("by block", 2100, 26, 2, 64, 64, 40, 2100, [2100]),     # 13 heads, more than 32 slots
]


@pytest.mark.parametrize("scales", ["free", "apart"])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("way,n,H,h,d,block,topk,max_kv,lens", CASES)
def test_paths(scales, paged, way, n, H, h, d, block, topk, max_kv, lens):
    assert q8_bounds.path(len(lens), n, H, h, d, block, topk, max_kv) == way
    g = gen(n + H * d + topk)
    c, table = filled(g, batch=len(lens), max_kv=max_kv, h=h, d=d, block=block, paged=paged,
                      scales=scales)
    q = rows(g, len(lens), n, H, d)
    ids = pick(g, lens, n, h, -(-max_kv // block), block, topk)
    ws = msa.Workspace(DEV)
    out, lse = msa.msa_sparse_attn_q8(
        q, c.k, c.v, c.k_scale, c.v_scale, ids, block=block, return_lse=True, block_table=table,
        seq_lens=torch.tensor(lens, dtype=torch.int32, device=DEV), max_kv=max_kv, workspace=ws)
    assert msa.msa_get_device_status(ws) == msa.MSA_OK
    check(c, table, q, ids, lens, block, max_kv, out, lse, way == "by block")


@pytest.mark.parametrize("H,d,block", [(8, 128, 64), (32, 64, 64), (32, 128, 128)])
def test_partial_outputs_keep_eleven_bits(H, d, block):
    """Two blocks a query whose values have opposite signs, as on the CPU in
    test_q8_bounds.py: partial outputs of eight bits would not pass."""
    g = gen(d + H)
    n, h, L = 1100, 4, 4 * block
    c, _ = filled(g, batch=1, max_kv=1152, h=h, d=d, block=block, paged=False, scales="free")
    mag = u8(c.v) & 0x7f
    sign = (torch.arange(1152, device=DEV) // block % 2 == 1)[None, :, None, None]
    u8(c.v).copy_(torch.where(sign, mag | 0x80, mag))
    c.k_scale.fill_(2.0 ** -9)
    q = rows(g, 1, n, H, d)
    pair = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device=DEV)
    ids = pair[torch.randint(0, 2, (1, n, h), device=DEV, generator=g)].contiguous()
    assert q8_bounds.path(1, n, H, h, d, block, 2, 1152) == "by block"
    out, lse = msa.msa_sparse_attn_q8(q, c.k, c.v, c.k_scale, c.v_scale, ids, block=block,
                                      return_lse=True)
    check(c, None, q, ids, [1152], block, 1152, out, lse, True)


@pytest.mark.parametrize("n", [1, 160, 1100])
def test_layouts_give_the_same_bits_by_row_and_by_block(n):
    g = gen(22)
    block, h, d, H, max_kv, lens = 64, 4, 64, 32, 1200, [1200, 1130]
    way = q8_bounds.path(2, n, H, h, d, block, 5, max_kv)
    assert way == {1: "streamed", 160: "by row", 1100: "by block"}[n]
    c, _ = filled(g, batch=2, max_kv=max_kv, h=h, d=d, block=block, paged=False, scales="free")
    q, ids = rows(g, 2, n, H, d), pick(g, lens, n, h, -(-max_kv // block), block, 5)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)

    def run(k, v, ks, vs, **kw):
        return msa.msa_sparse_attn_q8(q, k, v, ks, vs, ids, block=block, seq_lens=sl,
                                      return_lse=True, **kw)

    want = run(c.k, c.v, c.k_scale, c.v_scale)
    token_major = [u8(t).contiguous().view(F8) for t in (c.k, c.v)]
    nblk = -(-max_kv // block)
    table = torch.randperm(2 * nblk, device=DEV, generator=g).view(2, nblk).int()
    pool = msa.q8_cache(num_pages=2 * nblk, h=h, d=d, d_idx=32, block=block)
    for dst, src in ((pool.k, c.k), (pool.v, c.v)):
        full = torch.zeros((2, nblk * block, h, d), dtype=torch.uint8, device=DEV)
        full[:, :max_kv] = u8(src)
        u8(dst)[table.long().view(-1)] = full.view(2 * nblk, block, h, d)
    for dst, src in ((pool.k_scale, c.k_scale), (pool.v_scale, c.v_scale)):
        dst[table.long().view(-1)] = src.view(2 * nblk, h)
    for other in (run(*token_major, c.k_scale, c.v_scale),
                  run(pool.k, pool.v, pool.k_scale, pool.v_scale, block_table=table,
                      max_kv=max_kv)):
        assert all(torch.equal(a, b) for a, b in zip(want, other))


def test_replayed_errors_are_read_from_a_given_workspace():
    """A graph captured with a Workspace records a page outside the pool there."""
    g = gen(9)
    block, h, d, H = 64, 2, 64, 8
    c, table = filled(g, batch=1, max_kv=256, h=h, d=d, block=block, paged=True, scales="free")
    q = rows(g, 1, 1, H, d)
    ids = torch.tensor([0, 1], dtype=torch.int32, device=DEV).expand(1, 1, h, 2).contiguous()
    ws = msa.Workspace(DEV)

    def call():
        return msa.msa_sparse_attn_q8(q, c.k, c.v, c.k_scale, c.v_scale, ids, block=block,
                                      block_table=table, max_kv=256, workspace=ws)

    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    graph.replay()
    assert msa.msa_get_device_status(ws) == msa.MSA_OK
    good = table.clone()
    table[0, 1] = 10_000
    graph.replay()
    assert msa.msa_get_device_status(ws) == msa.MSA_ERR_DEVICE_ASSERT
    table.copy_(good)
    graph.replay()
    assert msa.msa_get_device_status(ws) == msa.MSA_OK
