"""The 8-bit KV cache against its definition in 64 bits (tests/q8_ref.py, where the
tolerances are derived): codes and scales of the write bit for bit, the read-back bit for
bit, block scores and attention within the bounds of their roundings."""

import random

import pytest
import torch

import q8_ref
from block_sparse_gqa_03_b200 import msa

pytestmark = pytest.mark.gpu
DEV = "cuda"
F8 = torch.float8_e4m3fn


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def rows(g, *shape, spread=0.0):
    x = torch.randn(shape, device=DEV, generator=g)
    if spread:
        x = x * torch.exp2((torch.rand(shape[:-1] + (1,), device=DEV, generator=g) - 0.5) * spread)
    return x.to(torch.bfloat16)


def u8(t):
    return t.view(torch.uint8)


def random_cache(g, *, batch, max_kv, h, d, d_idx, block, paged, nan_tail=None, spread=2):
    """A filled cache and its block table.  Codes of normal values; scales are powers of
    two that differ between blocks and heads.  ``nan_tail``: lengths past which every code
    is NaN (never to be read into a result)."""
    nblk = -(-max_kv // block)
    table = None
    if paged:
        n = batch * nblk + 3
        table = torch.randperm(n, device=DEV, generator=g)[:batch * nblk].view(batch, nblk).int()
        c = msa.q8_cache(num_pages=n, h=h, d=d, d_idx=d_idx, block=block, device=DEV)
    else:
        c = msa.q8_cache(batch=batch, max_kv=max_kv, h=h, d=d, d_idx=d_idx, block=block, device=DEV)
    for codes in (c.k, c.v, c.k_idx):
        x = torch.randn(codes.shape, device=DEV, generator=g) * 100
        codes.copy_(x.clamp(-448, 448).to(F8))
    for s in (c.k_scale, c.v_scale, c.k_idx_scale):
        e = torch.randint(-spread, spread + 1, s.shape, device=DEV, generator=g)
        s.copy_(torch.exp2(e - 7.0))
    if nan_tail is not None:
        for b, L in enumerate(nan_tail):
            for codes in (c.k, c.v, c.k_idx):
                raw = u8(codes)
                if paged:
                    beta = L // block
                    if beta < nblk:
                        raw[int(table[b, beta]), L % block:] = 0x7f
                        raw[table[b, beta + 1:].long()] = 0x7f
                else:
                    raw[b, L:] = 0x7f
    return c, table


def ids_for(g, lens, n, h, nblk, block, topk, causal=True):
    """Random distinct visible blocks, in random order, -1 anywhere."""
    out = torch.full((len(lens), n, h, topk), -1, dtype=torch.int32, device=DEV)
    key = torch.rand((len(lens), n, h, nblk), device=DEV, generator=g)
    key[..., :] = torch.where(torch.rand(key.shape, device=DEV, generator=g) < 0.8, key, -1.0)
    for b, L in enumerate(lens):
        see = (L + block - 1) // block
        key[b, :, :, see:] = -1.0
    k = min(topk, nblk)
    val, idx = key.topk(k, -1)
    idx = torch.where(val >= 0, idx, -1).int()
    perm = torch.randperm(topk, device=DEV, generator=g)[:k]
    out[..., perm] = idx
    return out


def ref_values(c, table, block, b, max_kv):
    """k, v [max_kv, h, d] and k_idx [max_kv, di] of sequence b in 64 bits."""
    k = q8_ref.values(u8(c.k), c.k_scale, block, b, max_kv, table)
    v = q8_ref.values(u8(c.v), c.v_scale, block, b, max_kv, table)
    ki = q8_ref.values(u8(c.k_idx).unsqueeze(2), c.k_idx_scale.unsqueeze(-1), block, b, max_kv,
                       table)
    return k, v, ki[:, 0]


def ok(ws):
    assert msa.msa_get_device_status(ws) == msa.MSA_OK


# ------------------------------------------------------------------------- write
def check_append(c, table, kn, vn, kin, lens, block, ws=None):
    want = [t.clone() for t in (u8(c.k), u8(c.v), u8(c.k_idx).unsqueeze(2))]
    scales = [t.double() for t in (c.k_scale, c.v_scale, c.k_idx_scale.unsqueeze(-1))]
    max_kv = None if table is None else table.shape[1] * block
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    own = ws or msa.Workspace(DEV)
    msa.msa_append_kv_q8(*c, kn, vn, kin, block=block, seq_lens=sl, block_table=table,
                         max_kv=max_kv, workspace=own)
    if ws is None:
        ok(own)
    for codes, sc, new in zip(want, scales, (kn, vn, kin.unsqueeze(2))):
        q8_ref.append_one(codes, sc, new.double(), lens, block, table)
    torch.cuda.synchronize()
    for name, a, b in zip(("k", "v", "k_idx"), (u8(c.k), u8(c.v), u8(c.k_idx).unsqueeze(2)), want):
        assert torch.equal(a, b), name
    for name, a, b in zip(("k", "v", "k_idx"), (c.k_scale, c.v_scale, c.k_idx_scale.unsqueeze(-1)),
                          scales):
        assert torch.equal(a.double(), b), name + " scale"


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("n,h,d,d_idx,block,max_kv,lens", [
    (1, 8, 128, 128, 64, 700, [700, 1, 333, 64, 65]),   # one row: first, middle and last of a block
    (1, 1, 64, 32, 16, 33, [33, 16, 17]),
    (5, 3, 64, 64, 16, 200, [200, 5, 21, 16]),          # across a block border, from position 0
    (130, 2, 128, 32, 128, 400, [400, 131, 257]),
    (301, 4, 128, 128, 32, 301, [301, 301]),            # a whole sequence
    (64, 2, 64, 64, 64, 129, [129, 64, 128]),
])
def test_append(paged, n, h, d, d_idx, block, max_kv, lens):
    g = gen(n * 7 + h)
    c, table = random_cache(g, batch=len(lens), max_kv=max_kv, h=h, d=d, d_idx=d_idx, block=block,
                            paged=paged)
    kn, vn = rows(g, len(lens), n, h, d, spread=6), rows(g, len(lens), n, h, d, spread=6)
    check_append(c, table, kn, vn, rows(g, len(lens), n, d_idx), lens, block)


def test_append_row_by_row_with_growing_rows():
    """Each row twice the one before: the scale of a block grows at every step, and the
    older rows are rounded again each time."""
    g = gen(3)
    block, h, d, di = 16, 2, 64, 32
    c, table = random_cache(g, batch=2, max_kv=40, h=h, d=d, d_idx=di, block=block, paged=True)
    for i in range(40):
        f = 2.0 ** (i % 23 - 11)
        kn, vn, kin = rows(g, 2, 1, h, d) * f, rows(g, 2, 1, h, d) / f, rows(g, 2, 1, di) * f
        check_append(c, table, kn, vn, kin, [i + 1, max(1, i // 2)], block)


def test_append_extremes():
    """Infinities saturate, NaN stays NaN and neither moves the scale; zeros and tiny rows
    take the smallest scale; the largest bf16 values fit."""
    block, h, d, di = 16, 4, 64, 32
    g = gen(4)
    c, _ = random_cache(g, batch=1, max_kv=16, h=h, d=d, d_idx=di, block=block, paged=False)
    kn = rows(g, 1, 3, h, d)
    kn[0, 0, 0, 3], kn[0, 1, 0, 5], kn[0, 2, 0, 7] = torch.inf, -torch.inf, torch.nan
    kn[0, :, 1] = 0
    kn[0, :, 2] = 2.0 ** -130
    kn[0, 1, 3, 9] = 3.3895313892515355e38
    kin = torch.full((1, 3, di), torch.nan, device=DEV, dtype=torch.bfloat16)
    check_append(c, None, kn, -kn, kin, [3], block)
    assert float(c.k_scale[0, 0, 1]) == 2.0 ** -100 and float(c.k_scale[0, 0, 3]) == 2.0 ** 120
    # codes on both sides of a border between two codes, and on it (ties to even)
    vals = torch.tensor([448, 17, 19, 18, 21, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, -17, -19.0])
    kn = torch.zeros((1, 1, h, d), dtype=torch.bfloat16, device=DEV)
    kn[0, 0, :, :10] = vals.to(DEV).bfloat16()
    check_append(c, None, kn, kn, kin[:, :1], [1], block)


def test_append_leaves_out_what_is_not_given():
    g = gen(5)
    c, _ = random_cache(g, batch=2, max_kv=64, h=2, d=64, d_idx=32, block=16, paged=False)
    before = [t.clone() for t in c]
    msa.msa_append_kv_q8(*c, None, rows(g, 2, 3, 2, 64), None, block=16)
    torch.cuda.synchronize()
    for i in (0, 2, 3, 5):
        assert torch.equal(u8(before[i]), u8(c[i])), i
    assert not torch.equal(u8(before[1]), u8(c.v))


def test_append_bad_inputs_are_recorded_and_not_written():
    g = gen(6)
    block, h, d, di = 16, 2, 64, 32
    c, table = random_cache(g, batch=3, max_kv=48, h=h, d=d, d_idx=di, block=block, paged=True)
    new = rows(g, 3, 2, h, d), rows(g, 3, 2, h, d), rows(g, 3, 2, di)
    ws = msa.Workspace(DEV)
    kw = dict(block=block, max_kv=48, workspace=ws)
    lens = torch.tensor([40, 20, 48], dtype=torch.int32, device=DEV)
    # a page outside the pool (sequence 0), a scale that is no power of two (sequence 2)
    bad = table.clone()
    bad[0, 2] = 10_000
    c.k_scale[int(table[2, 2]), 1] = 0.3
    before = [t.clone() for t in c]
    msa.msa_append_kv_q8(*c, *new, seq_lens=lens, block_table=bad, **kw)
    assert msa.msa_get_device_status(ws) == msa.MSA_ERR_DEVICE_ASSERT
    p0, p1, p2 = int(table[0, 2]), int(table[1, 1]), int(table[2, 2])
    assert torch.equal(u8(c.k[p0]), u8(before[0][p0]))          # nothing in sequence 0's page
    assert not torch.equal(u8(c.k[p1]), u8(before[0][p1]))      # sequence 1 written
    assert torch.equal(u8(c.k[p2, :, 1]), u8(before[0][p2, :, 1]))  # head 1 of sequence 2 not
    assert not torch.equal(u8(c.k[p2, :, 0]), u8(before[0][p2, :, 0]))
    # a sequence of one row to which two are appended: the first has no place
    msa.msa_append_kv_q8(*c, *new, seq_lens=torch.tensor([1, 20, 32], dtype=torch.int32,
                                                         device=DEV), block_table=table, **kw)
    assert msa.msa_get_device_status(ws) == msa.MSA_ERR_DEVICE_ASSERT
    p = int(table[0, 0])
    s = c.k_scale[p].double()
    want = q8_ref.encode(new[0][0, 1].double() / s[:, None])
    assert torch.equal(u8(c.k[p, 0]), want)


# -------------------------------------------------------------------- read back
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("n,base,h,d,d_idx,block,max_kv,lens", [
    (1, 0, 2, 64, 32, 16, 50, [50, 1, 0]),
    (37, 11, 3, 128, 128, 64, 300, [300, 40, 11, 12]),
    (300, 0, 8, 128, 64, 128, 300, [300, 129]),
    (100, 33, 4, 64, 64, 32, 133, [133, 64, 90]),
])
def test_read(paged, n, base, h, d, d_idx, block, max_kv, lens):
    g = gen(n + base)
    c, table = random_cache(g, batch=len(lens), max_kv=max_kv, h=h, d=d, d_idx=d_idx, block=block,
                            paged=paged, nan_tail=lens)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    outs = [torch.full((len(lens), n) + t, 7.0, dtype=torch.bfloat16, device=DEV)
            for t in ((h, d), (h, d), (d_idx,))]
    ws = msa.Workspace(DEV)
    got = msa.msa_read_kv_q8(*c, n=n, token_base=base, block=block, seq_lens=sl,
                             block_table=table, max_kv=max_kv, k_out=outs[0], v_out=outs[1],
                             k_idx_out=outs[2], workspace=ws)
    ok(ws)
    for b, L in enumerate(lens):
        live = max(0, min(L, base + n) - base)
        for x, ref in zip(got, ref_values(c, table, block, b, max_kv)):
            assert torch.equal(x[b, :live].double(), ref[base:base + live])
            assert bool((x[b, live:] == 7).all())  # past the end: as it was


def test_read_rounds_where_a_scale_is_no_power_of_two():
    g = gen(8)
    c, _ = random_cache(g, batch=2, max_kv=80, h=2, d=64, d_idx=32, block=16, paged=False)
    c.k_scale.copy_(torch.rand(c.k_scale.shape, device=DEV, generator=g) + 0.1)
    k, v, ki = msa.msa_read_kv_q8(*c, n=80, block=16)
    for b in range(2):
        rk, rv, rki = ref_values(c, None, 16, b, 80)
        # one fp32 and one bf16 rounding
        assert bool(((k[b].double() - rk).abs() <= rk.abs() * (2.0 ** -8 + 2.0 ** -23)).all())
        assert torch.equal(v[b].double(), rv) and torch.equal(ki[b].double(), rki)


# ----------------------------------------------------------------- block scores
SCORE_CASES = [
    # n, h, d_idx, block, max_kv, lens, causal
    (1, 8, 128, 64, 5000, [5000, 1, 0, 777], True),
    (1, 1, 32, 16, 100, [100, 16, 17], True),
    (1, 16, 64, 128, 1000, [1000, 129], True),
    (1, 3, 128, 32, 31, [31, 5], True),
    (1, 9, 32, 128, 300, [300, 0], True),
    (7, 2, 32, 16, 100, [100, 3, 0, 7], True),       # queries before the first token
    (150, 4, 64, 64, 400, [400, 150, 201], True),
    (33, 2, 128, 128, 300, [300, 299], False),
    (40, 1, 128, 32, 40, [40], True),
]


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("n,h,d_idx,block,max_kv,lens,causal", SCORE_CASES)
def test_block_scores(paged, n, h, d_idx, block, max_kv, lens, causal):
    g = gen(n * h + d_idx)
    c, table = random_cache(g, batch=len(lens), max_kv=max_kv, h=1, d=64, d_idx=d_idx, block=block,
                            paged=paged, nan_tail=lens)
    q = rows(g, len(lens), n, h, d_idx, spread=8)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    ws = msa.Workspace(DEV)
    got = msa.msa_block_scores_q8(q, c.k_idx, c.k_idx_scale, block=block, causal=causal,
                                  seq_lens=sl, block_table=table, max_kv=max_kv, workspace=ws)
    ok(ws)
    for b, L in enumerate(lens):
        _, _, key = ref_values(c, table, block, b, max_kv)
        want, mag = q8_ref.scores(q[b].double(), key, L, block, causal)
        x = got[b].double()
        assert torch.equal(torch.isneginf(x), torch.isneginf(want))
        fin = torch.isfinite(want)
        assert bool(((x - want).abs()[fin] <= mag[fin] * 2.0 ** -16).all())


# -------------------------------------------------------------------- attention
ATTN_CASES = [
    # n, H, h, d, block, topk, max_kv, lens, causal
    (1, 8, 1, 128, 64, 4, 500, [500, 1, 0, 64, 65], True),
    (1, 64, 8, 128, 64, 40, 5000, [5000, 3333, 17], True),
    (1, 6, 2, 64, 16, 8, 900, [900], True),
    (1, 16, 1, 64, 128, 3, 700, [700, 129], True),          # 16 heads a group
    (1, 27, 3, 128, 32, 5, 400, [400, 31], True),           # 9 heads a group
    (1, 5, 5, 64, 64, 300, 64 * 300, [64 * 300 - 3], True), # one head a group, long lists
    (4, 12, 4, 128, 64, 4, 300, [300, 2, 0], True),         # queries before the first token
    (20, 4, 2, 64, 32, 3, 120, [120, 64], False),
    (333, 20, 2, 64, 32, 6, 700, [700, 100, 333], True),    # one row per block of threads
    (400, 16, 2, 128, 16, 5, 400, [400], True),
    (300, 6, 2, 64, 64, 4, 300, [300, 299], True),
    (260, 32, 4, 128, 64, 6, 600, [600, 261, 100], True),
    (300, 16, 1, 128, 128, 3, 500, [500, 300], True),
    (310, 10, 2, 64, 128, 2, 310, [310, 77], False),
    (200, 48, 16, 128, 64, 3, 256, [256], True),
    # more than 4096 rows, gathered by block
    (540, 24, 8, 64, 64, 4, 600, [600, 541], True),
    (520, 8, 8, 128, 128, 2, 700, [700, 300], True),         # queries before the first token
    (4200, 6, 1, 64, 128, 2, 4200, [4200], False),
    (1100, 64, 4, 128, 64, 5, 1100, [1100], True),
    (700, 18, 2, 64, 64, 17, 2000, [2000, 1500, 700], True),
    (280, 32, 16, 128, 64, 3, 320, [300], True),
    # many sequences: one CTA per row, short and long lists, groups on both sides of 8
    (1, 16, 8, 64, 64, 3, 200, [200 - i for i in range(80)], True),
    (1, 24, 8, 128, 64, 20, 1500, [1500 - 19 * i for i in range(75)], True),
    (1, 48, 4, 128, 128, 9, 1300, [1300 - 8 * i for i in range(150)], True),
    (1, 12, 4, 64, 16, 70, 1200, [1200 - 7 * i for i in range(160)], True),
]


def check_attn(c, table, q, ids, lens, block, max_kv, out, lse, causal=True, scale=None):
    d = q.shape[-1]
    partials = q.shape[1] > 1 and block >= 64
    for b, L in enumerate(lens):
        k, v, _ = ref_values(c, table, block, b, max_kv)
        o, z, A, dx, total, N = q8_ref.attention(q[b].double(), k, v, ids[b], L, block,
                                                 scale or d ** -0.5, causal)
        x, y = out[b].double(), lse[b].double()
        assert torch.equal(torch.isneginf(y), torch.isneginf(z))
        bound = q8_ref.out_bound(o, A, dx, total, N, partials)
        err = (x - o).abs()
        assert bool((err <= bound).all()), "sequence %d: error %g, bound there %g" % (
            b, float((err - bound).max()), float(bound.flatten()[(err - bound).argmax()]))
        fin = torch.isfinite(z)
        assert bool(((y - z).abs()[fin] <= q8_ref.lse_bound(z, dx)[fin]).all())


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("n,H,h,d,block,topk,max_kv,lens,causal", ATTN_CASES)
def test_sparse_attn(paged, n, H, h, d, block, topk, max_kv, lens, causal):
    g = gen(n + H * d + topk)
    c, table = random_cache(g, batch=len(lens), max_kv=max_kv, h=h, d=d, d_idx=32, block=block,
                            paged=paged, nan_tail=lens)
    q = rows(g, len(lens), n, H, d, spread=2)
    nblk = -(-max_kv // block)
    ids = ids_for(g, lens, n, h, nblk, block, topk)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    ws = msa.Workspace(DEV)
    out = torch.full((len(lens), n, H, d), 9.0, dtype=torch.bfloat16, device=DEV)
    out, lse = msa.msa_sparse_attn_q8(q, c.k, c.v, c.k_scale, c.v_scale, ids, block=block,
                                      causal=causal, seq_lens=sl, return_lse=True, out=out,
                                      block_table=table, max_kv=max_kv, workspace=ws)
    ok(ws)
    check_attn(c, table, q, ids, lens, block, max_kv, out, lse, causal)


def test_sparse_attn_scales_far_apart_and_peaked_rows():
    """Blocks whose V scales differ by 2^60, the small ones holding all the probability,
    and scores large enough that single keys win."""
    g = gen(21)
    lens, block, h, d, H = [256, 250], 64, 2, 128, 8
    c, _ = random_cache(g, batch=2, max_kv=1200, h=h, d=d, d_idx=32, block=block, paged=False)
    c.k_scale.fill_(2.0 ** -7)
    c.k_scale[:, 1] = 1.0
    c.v_scale[:, 0], c.v_scale[:, 2] = 2.0 ** -40, 2.0 ** 20
    c.v_scale[:, 1], c.v_scale[:, 3] = 2.0 ** -30, 2.0 ** 10
    q = rows(g, 2, 1, H, d)
    ids = torch.tensor([3, 1, -1, 0], dtype=torch.int32, device=DEV).expand(2, 1, h, 4).contiguous()
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    for n in (1, 130, 1100):  # streamed, by row, by block
        qq, ii = q.expand(2, n, H, d).contiguous(), ids.expand(2, n, h, 4).contiguous()
        out, lse = msa.msa_sparse_attn_q8(qq, c.k, c.v, c.k_scale, c.v_scale, ii, block=block,
                                          seq_lens=sl, return_lse=True)
        check_attn(c, None, qq, ii, lens, block, 1200, out, lse)


@pytest.mark.parametrize("n", [1, 70, 280, 480])
def test_layouts_give_the_same_bits(n):
    """Token-major, head-major and padded caches, and pages, hold the same values."""
    g = gen(22)
    block, h, d, di, H, max_kv, lens = 64, 4, 128, 64, 16, 500, [500, 130]
    c, _ = random_cache(g, batch=2, max_kv=max_kv, h=h, d=d, d_idx=di, block=block, paged=False)
    q, qi = rows(g, 2, n, H, d), rows(g, 2, n, h, di)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    kw = dict(block=block, topk=5, seq_lens=sl, return_ids=True, return_scores=True,
              return_lse=True)

    def run(k, v, ki, ks, vs, kis, **more):
        r = msa.msa_forward_q8(q, k, v, qi, ki, ks, vs, kis, **kw, **more)
        torch.cuda.synchronize()
        return r

    want = run(*c)
    token_major = [u8(t).contiguous().view(F8) for t in c[:2]]
    wide = [torch.zeros((2, max_kv, h + 1, d + 16), dtype=torch.uint8, device=DEV) for _ in "kv"]
    for w, t in zip(wide, c[:2]):
        w[:, :, :h, :d] = u8(t)
    padded = [w[:, :, :h, :d].view(F8) for w in wide]
    nblk = -(-max_kv // block)
    table = torch.randperm(2 * nblk, device=DEV, generator=g).view(2, nblk).int()
    pool = msa.q8_cache(num_pages=2 * nblk, h=h, d=d, d_idx=di, block=block)
    for dst, src in zip(pool[:3], c[:3]):
        full = torch.zeros((2, nblk * block) + tuple(src.shape[2:]), dtype=torch.uint8, device=DEV)
        full[:, :max_kv] = u8(src)
        u8(dst)[table.long().view(-1)] = full.view((2 * nblk, block) + tuple(src.shape[2:]))
    for dst, src in zip(pool[3:], c[3:]):
        dst[table.long().view(-1)] = src.view((2 * nblk,) + tuple(src.shape[2:]))
    for other in (run(*token_major, *c[2:]), run(*padded, *c[2:]),
                  run(*pool, block_table=table, max_kv=max_kv)):
        for a, b in zip(want, other):
            assert torch.equal(a, b)


def test_bad_page_is_recorded_and_reads_as_zeros():
    g = gen(23)
    block, h, d, di, H, lens = 32, 2, 64, 64, 4, [128, 100]
    c, table = random_cache(g, batch=2, max_kv=128, h=h, d=d, d_idx=di, block=block, paged=True)
    bad = table.clone()
    bad[0, 1] = c.k.shape[0]
    bad[1, 2] = -5
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    ws = msa.Workspace(DEV)
    kw = dict(block=block, seq_lens=sl, block_table=bad, max_kv=128, workspace=ws)
    ids = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV).expand(2, 1, h, 3).contiguous()
    q, qi = rows(g, 2, 1, H, d), rows(g, 2, 1, h, di)
    got = msa.msa_block_scores_q8(qi, c.k_idx, c.k_idx_scale, **kw)
    assert msa.msa_get_device_status(ws) == msa.MSA_ERR_DEVICE_ASSERT
    assert bool((got[0, 0, :, 1] == 0).all()) and bool((got[1, 0, :, 2] == 0).all())
    out, lse = msa.msa_sparse_attn_q8(q, c.k, c.v, c.k_scale, c.v_scale, ids, return_lse=True, **kw)
    assert msa.msa_get_device_status(ws) == msa.MSA_ERR_DEVICE_ASSERT
    k, v, ki = msa.msa_read_kv_q8(*c, n=128, **kw)
    assert msa.msa_get_device_status(ws) == msa.MSA_ERR_DEVICE_ASSERT
    assert bool((k[0, 32:64] == 0).all()) and bool((ki[1, 64:96] == 0).all())
    # the values the read-back gives are those the attention saw
    for b, L in enumerate(lens):
        o, z, A, dx, total, N = q8_ref.attention(q[b].double(), k[b].double(), v[b].double(),
                                                 ids[b], L, block, d ** -0.5)
        assert bool(((out[b].double() - o).abs() <= q8_ref.out_bound(o, A, dx, total, N,
                                                                     False)).all())
    # a good table on the same workspace runs clean again
    msa.msa_sparse_attn_q8(q, c.k, c.v, c.k_scale, c.v_scale, ids, **dict(kw, block_table=table))
    ok(ws)


def test_ids_out_of_range_are_skipped_and_recorded():
    g = gen(24)
    block, h, d, H = 64, 1, 64, 4
    for n, max_kv in ((1, 700), (700, 700), (4200, 4200)):  # streamed, by row, by block
        c, _ = random_cache(g, batch=1, max_kv=max_kv, h=h, d=d, d_idx=32, block=block, paged=False)
        q = rows(g, 1, n, H, d)
        ids = torch.tensor([0, -(-max_kv // block), 2, 10], dtype=torch.int32, device=DEV)
        ids = ids.expand(1, n, h, 4).contiguous()
        ws = msa.Workspace(DEV)
        out, lse = msa.msa_sparse_attn_q8(q, c.k, c.v, c.k_scale, c.v_scale, ids, block=block,
                                          return_lse=True, workspace=ws)
        assert msa.msa_get_device_status(ws) == msa.MSA_ERR_DEVICE_ASSERT
        check_attn(c, None, q, ids, [max_kv], block, max_kv, out, lse)


# ------------------------------------------------------------- a run of them together
@pytest.mark.parametrize("paged,d,d_idx,block", [(False, 128, 128, 64), (True, 64, 32, 16)])
def test_prompt_then_steps(paged, d, d_idx, block):
    """A prompt is written and attended to, then tokens come one at a time: write, select,
    attend; at the end the cache is read back.  Every call against its definition on the
    cache as the calls before left it."""
    g = gen(31)
    batch, h, H, topk, max_kv, n0 = 2, 2, 8, 4, 400, 370
    nblk = -(-max_kv // block)
    if paged:
        table = torch.randperm(2 * nblk, device=DEV, generator=g).view(2, nblk).int()
        c = msa.q8_cache(num_pages=2 * nblk, h=h, d=d, d_idx=d_idx, block=block)
    else:
        table, c = None, msa.q8_cache(batch=2, max_kv=max_kv, h=h, d=d, d_idx=d_idx, block=block)
    ws = msa.Workspace(DEV)
    lens = [n0, n0]
    for n in [n0] + [1] * 20:
        new = rows(g, batch, n, h, d), rows(g, batch, n, h, d), rows(g, batch, n, d_idx)
        check_append(c, table, *new, lens, block, ws=ws)
        sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
        q, qi = rows(g, batch, n, H, d), rows(g, batch, n, h, d_idx)
        kw = dict(block=block, seq_lens=sl, block_table=table, max_kv=max_kv, workspace=ws)
        out, ids, scores, lse = msa.msa_forward_q8(
            q, c.k, c.v, qi, c.k_idx, c.k_scale, c.v_scale, c.k_idx_scale, topk=topk,
            force_own_block=True, return_ids=True, return_scores=True, return_lse=True, **kw)
        ids2 = msa.msa_index_select_q8(qi, c.k_idx, c.k_idx_scale, topk=topk,
                                       force_own_block=True, **kw)
        scores2 = msa.msa_block_scores_q8(qi, c.k_idx, c.k_idx_scale, **kw)
        out2, lse2 = msa.msa_sparse_attn_q8(q, c.k, c.v, c.k_scale, c.v_scale, ids,
                                            return_lse=True, **kw)
        ok(ws)
        assert torch.equal(ids, ids2) and torch.equal(scores, scores2)
        assert torch.equal(out, out2) and torch.equal(lse, lse2)
        check_attn(c, table, q, ids, lens, block, max_kv, out, lse)
        for b, L in enumerate(lens):  # ids: the best blocks by the scores, the own one first
            s = scores[b].clone()
            pos = (torch.arange(L - n, L, device=DEV) // block).view(n, 1, 1).expand(n, h, 1)
            s.scatter_(2, pos, torch.inf)
            best = s.sort(dim=-1, descending=True, stable=True)
            best = torch.where(best.values[..., :topk] > -torch.inf, best.indices[..., :topk], nblk)
            best = best.sort(-1).values
            assert torch.equal(torch.where(best == nblk, -1, best).int(), ids[b])
        lens = [x + 1 for x in lens]
    lens = [x - 1 for x in lens]
    got = msa.msa_read_kv_q8(*c, n=max_kv, **kw)
    for b, L in enumerate(lens):
        for x, ref in zip(got, ref_values(c, table, block, b, max_kv)):
            assert torch.equal(x[b, :L].double(), ref[:L])


def test_8bit_attention_is_the_bf16_attention_of_the_read_back_cache():
    """msa_sparse_attn on the read-back bf16 cache sees the same numbers: the two differ by
    their probabilities' rounding (bf16 there, f16 here) only."""
    g = gen(32)
    block, h, d, di, H, lens = 64, 2, 128, 64, 16, [900, 500]
    c, _ = random_cache(g, batch=2, max_kv=900, h=h, d=d, d_idx=di, block=block, paged=False,
                        spread=0)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    k, v, ki = msa.msa_read_kv_q8(*c, n=900, block=block, seq_lens=sl)
    for n, topk in ((1, 4), (400, 4), (900, 6)):  # streamed, by row, by block
        q, qi = rows(g, 2, n, H, d), rows(g, 2, n, h, di)
        kw = dict(block=block, seq_lens=sl)
        ids = msa.msa_index_select_q8(qi, c.k_idx, c.k_idx_scale, topk=topk, **kw)
        out, lse = msa.msa_sparse_attn_q8(q, c.k, c.v, c.k_scale, c.v_scale, ids, return_lse=True,
                                          **kw)
        out2, lse2 = msa.msa_sparse_attn(q, k, v, ids, return_lse=True, **kw)
        # |v| <= 448 * 2^-7: P rounded to 2^-8, outputs and partials to 2^-8, on either side
        assert bool(((out - out2).float().abs() <= 6 * 2.0 ** -8 * 3.5).all())
        fin = torch.isfinite(lse)
        assert torch.equal(fin, torch.isfinite(lse2))
        assert float((lse - lse2)[fin].abs().max()) <= 1e-3


# --------------------------------------------------------------- streams and graphs
def test_side_stream_and_captured_step():
    """A decode step (write, select, attend) captured once and replayed with new inputs
    gives the bits of eager calls; so does a run on a side stream."""
    g = gen(41)
    batch, block, h, d, di, H, topk, max_kv = 4, 64, 2, 128, 64, 16, 8, 1000

    def fresh():
        gg = gen(42)
        return random_cache(gg, batch=batch, max_kv=max_kv, h=h, d=d, d_idx=di, block=block,
                            paged=True)

    (c1, table), (c2, _) = fresh(), fresh()
    steps = [(rows(g, batch, 1, h, d), rows(g, batch, 1, h, d), rows(g, batch, 1, di),
              rows(g, batch, 1, H, d), rows(g, batch, 1, h, di)) for _ in range(4)]
    static = [t.clone() for t in steps[0]]
    lens = torch.tensor([700, 64, 1, 999], dtype=torch.int32, device=DEV)

    def step(c, kn, vn, kin, q, qi, ws):
        kw = dict(block=block, seq_lens=lens, block_table=table, max_kv=max_kv, workspace=ws)
        msa.msa_append_kv_q8(*c, kn, vn, kin, **kw)
        return msa.msa_forward_q8(q, c.k, c.v, qi, c.k_idx, c.k_scale, c.v_scale, c.k_idx_scale,
                                  topk=topk, return_ids=True, return_lse=True, **kw)

    ws1, ws2 = msa.Workspace(DEV), msa.Workspace(DEV)
    with pytest.raises(RuntimeError, match="cannot grow"):  # a workspace of the caller
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            step(c1, *static, msa.Workspace(DEV))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(c1, *static, ws1)  # warm-up: the same rows again at the same place
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step(c1, *static, ws1)
    # growing the workspace later must not pull the captured buffer away
    msa.msa_block_scores_q8(rows(g, 1, 300, 2, 64), msa.q8_cache(
        batch=1, max_kv=30000, h=2, d=64, d_idx=64, block=16).k_idx,
        torch.ones((1, 1875), device=DEV), block=16, workspace=ws1)
    with torch.cuda.stream(side):
        step(c2, *steps[0], ws2)
    side.synchronize()
    for s in steps:
        for a, b in zip(static, s):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            want = step(c2, *s, ws2)
        side.synchronize()
        for a, b in zip(res, want):
            assert torch.equal(a, b)
        for a, b in zip(c1, c2):
            assert torch.equal(u8(a), u8(b))
    ok(ws2)


def test_two_streams_at_once():
    """Calls on two streams with the default workspaces do not disturb each other."""
    g = gen(43)
    block, h, d, H, max_kv = 64, 4, 128, 32, 6000
    c, _ = random_cache(g, batch=2, max_kv=max_kv, h=h, d=d, d_idx=32, block=block, paged=False)
    nblk = -(-max_kv // block)
    qs = [rows(g, 2, 1, H, d) for _ in range(2)]
    ids = [ids_for(g, [max_kv] * 2, 1, h, nblk, block, 64) for _ in range(2)]

    def call(i):
        return msa.msa_sparse_attn_q8(qs[i], c.k, c.v, c.k_scale, c.v_scale, ids[i], block=block)

    want = [call(i).clone() for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(30):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(call(i))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in outs[i])


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("max_kv", [1024, 1000])
def test_scores_of_small_blocks_at_any_address(block, max_kv):
    """A prompt's scores are stored four blocks at a time where rows are 16-byte aligned:
    the same bits elsewhere, and nothing beside them."""
    g = gen(45)
    c, _ = random_cache(g, batch=2, max_kv=max_kv, h=3, d=64, d_idx=64, block=block, paged=False)
    lens = torch.tensor([max_kv, 417], dtype=torch.int32, device=DEV)
    qi = rows(g, 2, 150, 3, 64)
    nblk = -(-max_kv // block)
    kw = dict(block=block, seq_lens=lens)
    want = msa.msa_block_scores_q8(qi, c.k_idx, c.k_idx_scale, **kw)
    _, _, key = ref_values(c, None, block, 1, max_kv)
    ref, mag = q8_ref.scores(qi[1].double(), key, 417, block, True)
    fin = torch.isfinite(ref)
    assert torch.equal(torch.isneginf(want[1]), ~fin)
    assert bool(((want[1].double() - ref).abs()[fin] <= mag[fin] * 2.0 ** -16).all())
    for shift in (1, 2, 4):
        buf = torch.full((want.numel() + 8,), 7.0, device=DEV)
        part = buf[shift:shift + want.numel()].view(want.shape)
        msa.msa_block_scores_q8(qi, c.k_idx, c.k_idx_scale, block_scores=part, **kw)
        assert torch.equal(part, want) and part.shape[-1] == nblk
        assert bool((buf[:shift] == 7).all() and (buf[shift + want.numel():] == 7).all())


def test_stream_argument():
    """``stream=`` runs the call on that stream: its place in the order, its capture state
    and its allocations."""
    g = gen(44)
    block, h, d, H, max_kv = 64, 2, 64, 8, 3000
    c, _ = random_cache(g, batch=1, max_kv=max_kv, h=h, d=d, d_idx=32, block=block, paged=False)
    nblk = -(-max_kv // block)
    q = rows(g, 1, 1, H, d)
    ids = ids_for(g, [max_kv], 1, h, nblk, block, 32)

    def call(**kw):
        return msa.msa_sparse_attn_q8(q, c.k, c.v, c.k_scale, c.v_scale, ids, block=block, **kw)

    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = call(stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    out.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        call(stream=side, out=out)
        torch.cuda.current_stream().wait_stream(side)
    assert not out.any()  # captured, not run
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_cache_larger_than_32_bit_offsets():
    """2^31 codes and more in one tensor: the last row is written, scored, attended to and
    read back."""
    g = gen(51)
    block, h, d, di, H, max_kv = 64, 8, 128, 128, 16, (1 << 21) + 130
    c = msa.q8_cache(batch=1, max_kv=max_kv, h=h, d=d, d_idx=di, block=block)
    assert c.k.numel() > 1 << 31
    n, last = 70, (max_kv - 1) // block
    new = rows(g, 1, n, h, d), rows(g, 1, n, h, d), rows(g, 1, n, di)
    ws = msa.Workspace(DEV)
    msa.msa_append_kv_q8(*c, *new, block=block, workspace=ws)
    k, v, ki = msa.msa_read_kv_q8(*c, n=n, token_base=max_kv - n, block=block, workspace=ws)
    for got, want in zip((k, v), new):
        assert bool(((got - want).abs() <= want.abs() * 2.0 ** -4 + 2.0 ** -8).all())
    q, qi = rows(g, 1, 1, H, d), rows(g, 1, 1, h, di)
    ids = torch.tensor([last, last - 1], dtype=torch.int32, device=DEV).expand(1, 1, h, 2).contiguous()
    out, lse = msa.msa_sparse_attn_q8(q, c.k, c.v, c.k_scale, c.v_scale, ids, block=block,
                                      return_lse=True, workspace=ws)
    ok(ws)
    base = (last - 1) * block
    local = torch.tensor([1, 0], dtype=torch.int32, device=DEV).expand(1, h, 2)
    kk, vv, _ = msa.msa_read_kv_q8(*c, n=max_kv - base, token_base=base, block=block)
    o, z, A, dx, total, N = q8_ref.attention(q[0].double(), kk[0].double(), vv[0].double(), local,
                                             max_kv - base, block, d ** -0.5)
    assert bool(((out[0].double() - o).abs() <= q8_ref.out_bound(o, A, dx, total, N, False)).all())
    assert bool(((lse[0].double() - z).abs() <= q8_ref.lse_bound(z, dx)).all())
    s = msa.msa_block_scores_q8(qi, c.k_idx, c.k_idx_scale, block=block)
    want, mag = q8_ref.scores(qi[0].double(), ki[0].double()[-(max_kv - last * block):],
                              max_kv - last * block, block)
    assert bool(((s[0, 0, :, last].double() - want[0, :, 0]).abs() <= mag[0, :, 0] * 2.0 ** -16).all())


def test_codes_as_bytes_and_a_padded_index_key():
    """uint8 tensors hold the same codes; index-key rows may lie apart."""
    g = gen(52)
    c, _ = random_cache(g, batch=2, max_kv=200, h=2, d=64, d_idx=64, block=32, paged=False)
    wide = torch.zeros((2, 200, 96), dtype=torch.uint8, device=DEV)
    wide[:, :, :64] = u8(c.k_idx)
    q, ids = rows(g, 2, 1, 4, 64), ids_for(g, [200, 200], 1, 2, 7, 32, 3)
    for n in (1, 20):
        qi = rows(g, 2, n, 2, 64)
        want = msa.msa_block_scores_q8(qi, c.k_idx, c.k_idx_scale, block=32)
        got = msa.msa_block_scores_q8(qi, wide[:, :, :64], c.k_idx_scale, block=32)
        assert torch.equal(want, got)
    want = msa.msa_sparse_attn_q8(q, c.k, c.v, c.k_scale, c.v_scale, ids, block=32)
    got = msa.msa_sparse_attn_q8(q, u8(c.k), u8(c.v), c.k_scale, c.v_scale, ids, block=32)
    assert torch.equal(want, got)


def test_refusals_name_the_argument():
    g = gen(53)
    c, table = random_cache(g, batch=2, max_kv=64, h=2, d=64, d_idx=32, block=16, paged=False)
    q, ids = rows(g, 2, 1, 4, 64), torch.zeros((2, 1, 2, 3), dtype=torch.int32, device=DEV)
    new = rows(g, 2, 1, 2, 64)
    a = [q, c.k, c.v, c.k_scale, c.v_scale, ids]
    for i, bad, word in ((0, q.float(), "q"), (0, rows(g, 3, 1, 4, 64), "sequences"),
                         (1, c.k.float(), "k"), (2, c.v[:, :, :1], "v"),
                         (3, c.k_scale.half(), "k_scale"), (4, c.v_scale[:, :-1], "v_scale"),
                         (5, ids.long(), "block_ids"), (5, ids[:, :, :1], "block_ids")):
        args = list(a)
        args[i] = bad
        with pytest.raises(ValueError, match=word):
            msa.msa_sparse_attn_q8(*args, block=16)
    with pytest.raises(ValueError, match="seq_lens"):
        msa.msa_sparse_attn_q8(*a, block=16, seq_lens=torch.zeros(2, device=DEV))
    with pytest.raises(ValueError, match="k_new"):
        msa.msa_append_kv_q8(*c, new.transpose(2, 3), block=16)
    with pytest.raises(ValueError, match="max_kv"):
        msa.msa_append_kv_q8(*c, new, block=16, max_kv=63)
    with pytest.raises(ValueError, match="max_kv"):
        msa.msa_append_kv_q8(*c, new, block=16, block_table=torch.zeros((2, 4), dtype=torch.int32,
                                                                       device=DEV))
    with pytest.raises(ValueError, match="page"):  # the pool's pages are not of `block` tokens
        msa.msa_append_kv_q8(*c, new, block=16, max_kv=64,
                             block_table=torch.zeros((2, 4), dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError, match="rows"):
        msa.msa_read_kv_q8(*c, n=3, block=16, k_out=new, v_out=new, k_idx_out=new)
    with pytest.raises(msa.MsaError):
        msa.msa_read_kv_q8(*c, n=10, token_base=60, block=16)
    with pytest.raises(msa.MsaError):  # strides of 24 bytes
        msa.msa_block_scores_q8(rows(g, 2, 1, 1, 32), torch.zeros(
            (2, 64, 40), dtype=torch.uint8, device=DEV)[:, :, :32], c.k_idx_scale, block=16)


# ------------------------------------------------------------------- random shapes
@pytest.mark.parametrize("seed", range(24))
def test_random_shapes(seed):
    r = random.Random(seed)
    g = gen(100 + seed)
    block, d, di = r.choice((16, 32, 64, 128)), r.choice((64, 128)), r.choice((32, 64, 128))
    h, G, batch = r.choice((1, 2, 3, 5)), r.randint(1, 16), r.randint(1, 3)
    max_kv = r.randint(1, 900)
    n = 1 if r.random() < 0.5 else r.randint(1, max_kv)
    topk, paged, causal = r.randint(1, 9), r.random() < 0.5, r.random() < 0.8
    H = h * G
    lens = [r.randint(n, max_kv) for _ in range(batch)]
    c, table = random_cache(g, batch=batch, max_kv=max_kv, h=h, d=d, d_idx=di, block=block,
                            paged=paged, nan_tail=lens)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    kn, vn, kin = rows(g, batch, n, h, d), rows(g, batch, n, h, d), rows(g, batch, n, di)
    check_append(c, table, kn, vn, kin, lens, block)
    q, qi = rows(g, batch, n, H, d), rows(g, batch, n, h, di)
    kw = dict(block=block, seq_lens=sl, block_table=table, max_kv=max_kv, causal=causal)
    ws = msa.Workspace(DEV)
    out, ids, scores, lse = msa.msa_forward_q8(
        q, c.k, c.v, qi, c.k_idx, c.k_scale, c.v_scale, c.k_idx_scale, topk=topk, return_ids=True,
        return_scores=True, return_lse=True, workspace=ws, **kw)
    ok(ws)
    for b, L in enumerate(lens):
        _, _, key = ref_values(c, table, block, b, max_kv)
        want, mag = q8_ref.scores(qi[b].double(), key, L, block, causal)
        x = scores[b].double()
        assert torch.equal(torch.isneginf(x), torch.isneginf(want))
        fin = torch.isfinite(want)
        assert bool(((x - want).abs()[fin] <= mag[fin] * 2.0 ** -16).all())
    check_attn(c, table, q, ids, lens, block, max_kv, out, lse, causal)
