"""Which workspace a call takes when it is given none."""

import types

import pytest
import torch

from block_sparse_gqa_03_b200 import msa


def test_8bit_calls_on_any_stream_share_none_with_the_bf16_calls(monkeypatch):
    """A bf16 call on a side stream and an 8-bit call on the default one may run at once."""
    taken = []
    like = types.SimpleNamespace(get_device=lambda: 0, device=torch.device("cuda", 0))
    stream = {"raw": 0}
    monkeypatch.setattr(msa, "_default_ws", {})
    monkeypatch.setattr(msa, "_get_device", lambda: 0)
    monkeypatch.setattr(msa, "_raw_stream", lambda dev: stream["raw"])
    monkeypatch.setattr(msa, "_capturing", lambda: False)

    class Marshal:
        @staticmethod
        def index(buffer, raw):
            taken.append(buffer)
            return msa.MSA_OK

    class Space:
        def __init__(self, device):
            self.buf = self

    monkeypatch.setattr(msa, "_marshal", Marshal)
    monkeypatch.setattr(msa, "Workspace", Space)
    shared = msa._workspace(None, like.device)
    for raw in (0, 64, 0, 128):
        stream["raw"] = raw
        msa._run_q8("msa_block_scores_q8", "index", like, None, ())
    assert all(t is not shared for t in taken)
    assert taken[0] is taken[2] and len({id(t) for t in taken}) == 3


@pytest.mark.gpu
def test_mixed_calls_on_two_streams():
    """The bf16 selection of one stream beside 8-bit attention with split rows on another."""
    g = torch.Generator(device="cuda").manual_seed(3)
    block, h, d, H, max_kv = 64, 4, 128, 32, 6000

    def draw(*shape):
        return torch.randn(shape, device="cuda", generator=g).to(torch.bfloat16)

    c = msa.q8_cache(batch=2, max_kv=max_kv, h=h, d=d, d_idx=64, block=block)
    msa.msa_append_kv_q8(*c, draw(2, max_kv, h, d), draw(2, max_kv, h, d), draw(2, max_kv, 64),
                         block=block)
    k, v, ki = msa.msa_read_kv_q8(*c, n=max_kv, block=block)
    q, qi = draw(2, 1, H, d), draw(2, 1, h, 64)

    def one(stream=None):
        ids = msa.msa_index_select(qi, ki, block=block, topk=64, stream=stream)
        return ids, msa.msa_sparse_attn(q, k, v, ids, block=block, stream=stream)

    def eight():
        return msa.msa_forward_q8(q, c.k, c.v, qi, c.k_idx, c.k_scale, c.v_scale, c.k_idx_scale,
                                  block=block, topk=64, return_ids=True)

    want1, want8 = [t.clone() for t in one()], [t.clone() for t in eight()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    runs = [(one(side), eight()) for _ in range(30)]
    torch.cuda.synchronize()
    for a, b in runs:
        assert all(torch.equal(x, y) for x, y in zip(a, want1))
        assert all(torch.equal(x, y) for x, y in zip(b, want8))
