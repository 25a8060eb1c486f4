"""The 8-bit cache's calls on a machine without a GPU: bad arguments are refused on the
host before anything is launched, workspace sizes and launch counts, and the tests' own
e4m3 table against torch's conversion."""

import ctypes

import pytest
import torch

import q8_ref
from block_sparse_gqa_03_b200 import build as msa_build
from block_sparse_gqa_03_b200 import msa

FAKE = 1 << 20  # an aligned address that is never dereferenced: validation fails first
SB = 4096


@pytest.fixture(scope="module")
def lib():
    msa_build.build()
    return msa.load_library()


def params(**kw):
    base = dict(batch=2, n_q=1, max_kv=1024, H=8, h=2, d=128, d_idx=64, block=64, topk=4)
    base.update(kw)
    p = msa.make_params(**base)
    h, d, di, n = base["h"], base["d"], base["d_idx"], base["n_q"]
    p.q_strides[:] = [n * base["H"] * d, base["H"] * d, d]
    p.o_strides[:] = p.q_strides[:]
    p.k_strides[:] = [1024 * h * d, h * d, d]
    p.v_strides[:] = p.k_strides[:]
    p.qi_strides[:] = [n * h * di, h * di, di]
    p.ki_strides[:] = [1024 * di, di]
    return p


def append(lib, p, kn=FAKE, vn=FAKE, kin=FAKE, k=FAKE, v=FAKE, ki=FAKE, ks=FAKE, vs=FAKE,
           kis=FAKE, ws=FAKE, nb=SB):
    return lib.msa_append_kv_q8(ctypes.byref(p), kn, vn, kin, k, v, ki, ks, vs, kis, ws, nb, None)


def read(lib, p, base=0, k=FAKE, v=FAKE, ki=FAKE, ks=FAKE, vs=FAKE, kis=FAKE, ko=FAKE, vo=FAKE,
         kio=FAKE, ws=FAKE, nb=SB):
    return lib.msa_read_kv_q8(ctypes.byref(p), k, v, ki, ks, vs, kis, base, ko, vo, kio, ws, nb,
                              None)


def test_append_refusals(lib):
    bad, small = msa.MSA_ERR_INVALID_ARG, msa.MSA_ERR_WORKSPACE
    p = params()
    assert append(lib, p, kn=None, vn=None, kin=None) == bad  # nothing to write
    for name in ("k", "v", "ki", "ks", "vs", "kis"):
        assert append(lib, p, **{name: None}) == bad, name
    for name, off in (("kn", 2), ("vn", 8), ("kin", 8), ("k", 8), ("v", 1), ("ki", 4), ("ks", 2)):
        assert append(lib, p, **{name: FAKE + off}) == bad, name
    assert append(lib, p, nb=SB - 1) == small
    assert append(lib, p, ws=FAKE + 16) == small
    assert append(lib, p, ws=None) == small
    for field, axis in (("k_strides", 0), ("k_strides", 1), ("v_strides", 2), ("ki_strides", 1)):
        q = params()
        getattr(q, field)[axis] += 8  # a multiple of 8, not of 16
        assert append(lib, q) == bad, field
    q = params()
    q.k_strides[2] = 64  # heads closer than d
    assert append(lib, q) == bad
    assert append(lib, params(n_q=2048)) == bad  # more rows than the cache holds
    assert append(lib, params(d=96)) == msa.MSA_ERR_UNSUPPORTED


def test_read_refusals(lib):
    bad = msa.MSA_ERR_INVALID_ARG
    p = params(n_q=24)
    assert read(lib, p, base=-1) == bad
    assert read(lib, p, base=1001) == bad  # 1001 + 24 > 1024
    assert read(lib, p, ko=None, vo=None, kio=None) == bad
    assert read(lib, p, kis=None) == bad
    assert read(lib, p, vo=FAKE + 8) == bad
    assert read(lib, p, nb=100) == msa.MSA_ERR_WORKSPACE


def test_score_and_attention_refusals(lib):
    bad, small = msa.MSA_ERR_INVALID_ARG, msa.MSA_ERR_WORKSPACE
    p = params()
    byref = ctypes.byref

    def sc(q=FAKE, k=FAKE, s=FAKE, out=FAKE, nb=1 << 40, p=p):
        return lib.msa_block_scores_q8(byref(p), q, k, s, out, FAKE, nb, None)

    assert sc(q=None) == bad and sc(k=None) == bad and sc(s=None) == bad and sc(out=None) == bad
    assert sc(q=FAKE + 8) == bad and sc(k=FAKE + 8) == bad and sc(s=FAKE + 1) == bad
    assert sc(nb=SB - 1) == small
    many = params(n_q=16)
    need = msa.msa_workspace_size(many, msa.MSA_OP_BLOCK_SCORES_Q8)
    assert need >= SB + 2 * 1024 * 64 * 2  # the widened index key
    assert sc(p=many, nb=need - 1) == small
    assert lib.msa_index_select_q8(byref(p), FAKE, FAKE, FAKE, None, None, FAKE, 1 << 40,
                                   None) == bad

    def at(q=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, ids=FAKE, out=FAKE, nb=1 << 40, p=p):
        return lib.msa_sparse_attn_q8(byref(p), q, k, v, ks, vs, ids, out, None, FAKE, nb, None)

    for name in ("q", "k", "v", "ks", "vs", "ids", "out"):
        assert at(**{name: None}) == bad, name
    for name in ("q", "k", "v", "out"):
        assert at(**{name: FAKE + 8}) == bad, name
    need = msa.msa_workspace_size(p, msa.MSA_OP_SPARSE_ATTN_Q8)
    assert need >= SB and at(nb=need - 1) == small
    q = params()
    q.o_strides[1] += 4
    assert at(p=q) == bad

    def fw(**kw):
        a = dict(q=FAKE, k=FAKE, v=FAKE, qi=FAKE, ki=FAKE, ks=FAKE, vs=FAKE, kis=FAKE, out=FAKE)
        a.update(kw)
        return lib.msa_forward_q8(byref(p), *a.values(), None, None, None, FAKE, 64, None)

    for name in ("q", "k", "v", "qi", "ki", "ks", "vs", "kis", "out"):
        assert fw(**{name: None}) == bad, name
    assert fw() == small


def test_launch_counts_and_sizes(lib):
    one, many = params(), params(n_q=16)
    count = msa.msa_launch_count
    assert count(one, msa.MSA_OP_APPEND_KV_Q8) == count(one, msa.MSA_OP_READ_KV_Q8) == 1
    assert count(one, msa.MSA_OP_BLOCK_SCORES_Q8) == 1
    assert count(many, msa.MSA_OP_BLOCK_SCORES_Q8) == 2
    assert count(one, msa.MSA_OP_FORWARD_Q8) == 2 + count(one, msa.MSA_OP_SPARSE_ATTN_Q8)
    for op in (msa.MSA_OP_APPEND_KV_Q8, msa.MSA_OP_READ_KV_Q8, msa.MSA_OP_BLOCK_SCORES_Q8):
        assert msa.msa_workspace_size(one, op) == msa.STATUS_BYTES
    assert msa.msa_workspace_size(params(block=48), msa.MSA_OP_FORWARD_Q8) == 0


def test_binding_refuses_cpu_tensors_and_bad_geometry():
    c = msa.q8_cache(batch=1, max_kv=64, h=2, d=64, d_idx=32, block=16, device="cpu")
    new = torch.zeros((1, 1, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        msa.msa_append_kv_q8(*c, new, block=16)
    with pytest.raises(ValueError, match="no new rows"):
        msa.msa_append_kv_q8(*c, block=16)
    with pytest.raises(ValueError):
        msa.q8_cache(h=2, d=64, d_idx=32, block=16, device="cpu")
    assert c.k.shape == (1, 64, 2, 64) and c.k_scale.shape == (1, 4, 2)
    pool = msa.q8_cache(num_pages=5, h=2, d=64, d_idx=32, block=16, device="cpu")
    assert pool.v.shape == (5, 16, 2, 64) and pool.k_idx_scale.shape == (5,)


def test_binding_fails_loudly_without_its_extension(lib, monkeypatch):
    monkeypatch.setattr(msa, "MARSHAL_PATH", "/nonexistent/_marshal.so")
    with pytest.raises(RuntimeError, match="not built"):
        msa._marshal_module()


def test_marshalling_refuses_what_is_no_tensor(lib):
    m = msa._marshal_module()
    with pytest.raises(ValueError, match="arguments"):
        m.attn(1, 2)
    with pytest.raises(ValueError, match="must be a tensor"):
        m.index(*range(13))
    x = torch.zeros((1, 1, 1, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        m.attn(x, x, x, x, x, x, x, None, True, 0.0, 64, None, None, None, None, 0)


def test_reference_table_and_rounding():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double()
    assert torch.equal(torch.nan_to_num(q8_ref.decode(codes)), torch.nan_to_num(want))
    assert torch.equal(torch.isnan(q8_ref.decode(codes)), torch.isnan(want))
    g = torch.Generator().manual_seed(1)
    x = torch.randn(20000, generator=g) * torch.exp2(torch.rand(20000, generator=g) * 20 - 12)
    x = torch.cat([x.clamp(-448, 448), torch.tensor([0.0, -0.0, 448.0, 2.0 ** -10, 3 * 2.0 ** -10,
                                                     -(2.0 ** -10), 17.0, 19.0, 432.0])])
    got = q8_ref.encode(x.double())
    assert torch.equal(got, x.to(torch.float8_e4m3fn).view(torch.uint8))
    assert q8_ref.scale_for(448.0) == 1.0 and q8_ref.scale_for(449.0) == 2.0
    assert q8_ref.scale_for(0.0) == 2.0 ** -100
