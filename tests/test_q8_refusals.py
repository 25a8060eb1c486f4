"""Arguments of the 8-bit cache's calls at the ends of their types, and the workspaces that
large capacities ask for (no GPU needed: nothing is launched)."""

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


def test_workspace_of_scores_does_not_grow_with_batch_times_capacity(lib):
    """64 sequences in pages, each of up to 1M tokens, two queries a sequence: the lengths
    are on the device, so only the capacity is known.  Beside the scores (64 x 2 x 8 x 16384
    fp32 for a selection) the workspace holds a part of the index keys."""
    p = params(batch=64, n_q=2, max_kv=1 << 20, H=8, h=8, d_idx=128)
    slack = 1 << 24  # scales, alignment, ids
    assert msa.msa_workspace_size(p, msa.MSA_OP_BLOCK_SCORES_Q8) <= (1 << 30) + slack
    scores = 64 * 2 * 8 * 16384 * 4
    assert msa.msa_workspace_size(p, msa.MSA_OP_INDEX_SELECT_Q8) <= (1 << 30) + scores + slack
    assert msa.msa_launch_count(p, msa.MSA_OP_BLOCK_SCORES_Q8) == 32  # four sequences at a time
    assert msa.msa_launch_count(p, msa.MSA_OP_INDEX_SELECT_Q8) == 33
    one = params(batch=1, n_q=2, max_kv=65536 * 128, block=128, d_idx=128)  # the longest there is
    assert msa.msa_workspace_size(one, msa.MSA_OP_BLOCK_SCORES_Q8) <= 2 * one.max_kv * 128 + slack
    assert msa.msa_launch_count(one, msa.MSA_OP_BLOCK_SCORES_Q8) == 2
