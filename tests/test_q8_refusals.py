"""Arguments of the 8-bit cache's calls at the ends of their types (no GPU needed: they are
refused before anything is launched)."""

import ctypes

import pytest

from block_sparse_gqa_03_b200 import build as msa_build
from block_sparse_gqa_03_b200 import msa

FAKE = 1 << 20  # an aligned address that is never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    msa_build.build()
    return msa.load_library()


def params(**kw):
    base = dict(batch=2, n_q=24, max_kv=1024, H=8, h=2, d=128, d_idx=64, block=64, topk=4)
    base.update(kw)
    p = msa.make_params(**base)
    p.k_strides[:] = [1024 * 256, 256, 128]
    p.v_strides[:] = p.k_strides[:]
    p.ki_strides[:] = [1024 * 64, 64]
    return p


@pytest.mark.parametrize("base", [1001, 2**31 - 1, 2**31, 2**63 - 1, 2**63 - 24, 2**63 - 25, -1,
                                  -2**63])
def test_read_refuses_a_base_past_the_capacity(lib, base):
    rc = lib.msa_read_kv_q8(ctypes.byref(params()), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, base, FAKE,
                            FAKE, FAKE, FAKE, 4096, None)
    assert rc == msa.MSA_ERR_INVALID_ARG
