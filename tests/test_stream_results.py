"""``stream=`` of the calls: what a call allocates, fills and launches belongs to that
stream, so that work queued on the caller's own stream cannot overwrite its results."""

import contextlib
import types

import pytest
import torch

from block_sparse_gqa_03_b200 import msa

BF16, F8 = torch.bfloat16, torch.float8_e4m3fn


class Recording(torch.Tensor):
    """A CPU tensor that notes on which stream zeros of its kind are made."""

    log: list = []
    current = None

    def new_zeros(self, *a, **k):
        Recording.log.append(("zeros", Recording.current))
        return torch.zeros(*a, **k)


@pytest.fixture
def streams(monkeypatch):
    """A stand-in stream for CPU tensors, and the log of allocations and launches."""
    log = Recording.log = []
    Recording.current = None

    @contextlib.contextmanager
    def stream(s):
        before, Recording.current = Recording.current, s
        yield
        Recording.current = before

    def empty(like, lead, last=-1, kind=0):
        log.append(("empty", Recording.current))
        shape = tuple(like.shape[:lead]) + ((last,) if last >= 0 else ())
        return torch.empty(shape, dtype=(like.dtype, torch.float32, torch.int32)[kind])

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(msa, "_empty", empty)
    monkeypatch.setattr(msa, "_run_q8", lambda *a: log.append((a[0], Recording.current)))
    side = types.SimpleNamespace(device=types.SimpleNamespace(index=-1), cuda_stream=5)
    return side, log


def cache_and_rows():
    c = msa.q8_cache(batch=1, max_kv=64, h=2, d=64, d_idx=32, block=16, device="cpu")
    k = c.k.as_subclass(Recording)
    q, qi = torch.zeros((1, 1, 4, 64), dtype=BF16), torch.zeros((1, 1, 2, 32), dtype=BF16)
    return c._replace(k=k), q, qi


Q8_CALLS = {
    "append": lambda c, q, qi, **kw: msa.msa_append_kv_q8(
        *c, torch.zeros((1, 1, 2, 64), dtype=BF16), block=16, **kw),
    "read": lambda c, q, qi, **kw: msa.msa_read_kv_q8(*c, n=8, block=16, **kw),
    "scores": lambda c, q, qi, **kw: msa.msa_block_scores_q8(qi, c.k_idx, c.k_idx_scale, block=16,
                                                             **kw),
    "select": lambda c, q, qi, **kw: msa.msa_index_select_q8(qi, c.k_idx, c.k_idx_scale, block=16,
                                                             topk=2, return_scores=True, **kw),
    "attn": lambda c, q, qi, **kw: msa.msa_sparse_attn_q8(
        q, c.k, c.v, c.k_scale, c.v_scale, torch.zeros((1, 1, 2, 1), dtype=torch.int32), block=16,
        return_lse=True, **kw),
    "forward": lambda c, q, qi, **kw: msa.msa_forward_q8(
        q, c.k, c.v, qi, c.k_idx, c.k_scale, c.v_scale, c.k_idx_scale, block=16, topk=2,
        return_ids=True, return_scores=True, return_lse=True, **kw),
}
MADE = {"append": 0, "read": 3, "scores": 1, "select": 2, "attn": 2, "forward": 4}


@pytest.mark.parametrize("name", sorted(Q8_CALLS))
def test_results_are_made_on_the_calls_stream(name, streams):
    side, log = streams
    Q8_CALLS[name](*cache_and_rows(), stream=side)
    assert len(log) == MADE[name] + 1 and log[-1][0].startswith("msa_")
    assert all(s is side for _, s in log), log
    log.clear()
    Q8_CALLS[name](*cache_and_rows())  # without one: the current stream
    assert len(log) == MADE[name] + 1 and all(s is None for _, s in log)


@pytest.mark.parametrize("name", sorted(Q8_CALLS))
def test_a_stream_of_another_device_is_refused(name, streams):
    side, log = streams
    side.device.index = 3
    with pytest.raises(ValueError, match="stream"):
        Q8_CALLS[name](*cache_and_rows(), stream=side)
    assert not log


def bf16_calls():
    """The bf16 calls with everything left to them, by name: (call, results they make)."""
    def z(*shape, dtype=BF16):
        return torch.zeros(shape, dtype=dtype)

    q, qi = z(1, 1, 4, 64), z(1, 1, 2, 32)
    k, ki, ids = z(1, 64, 2, 64), z(1, 64, 32), z(1, 1, 2, 1, dtype=torch.int32)
    sel = dict(block=16, topk=2)
    return {
        "index_select": (lambda **kw: msa.msa_index_select(qi, ki, return_scores=True, **sel, **kw), 2),
        "index_topk": (lambda **kw: msa.msa_index_topk(qi, ki, return_scores=True, **sel, **kw), 2),
        "block_scores": (lambda **kw: msa.msa_block_scores(qi, ki, block=16, **kw), 1),
        "index_candidates": (lambda **kw: msa.msa_index_candidates(qi, ki, **sel, **kw), 2),
        "select_candidates": (lambda **kw: msa.msa_select_candidates(
            z(1, 1, 1, 2, 2, dtype=torch.float32), z(1, 1, 1, 2, 2, dtype=torch.int32), max_kv=64,
            want_local=True, **sel, **kw), 2),
        "sparse_attn": (lambda **kw: msa.msa_sparse_attn(q, k, k, ids, block=16, return_lse=True,
                                                         **kw), 2),
        "sparse_attn_noalloc": (lambda **kw: msa.msa_sparse_attn_noalloc(q, k, k, ids, block=16,
                                                                         **kw), 1),
        "append_kv": (lambda **kw: msa.msa_append_kv(k, k, ki, k[:, :1], None, None, block=16,
                                                     **kw), 0),
        "append_kv_values": (lambda **kw: msa.msa_append_kv(None, k, ki, None, k[:, :1], None,
                                                            block=16, **kw), 0),
        "merge_partials": (lambda **kw: msa.msa_merge_partials(
            z(2, 1, 1, 4, 64), z(2, 1, 1, 4, dtype=torch.float32), **kw), 1),
        "shard_lengths": (lambda **kw: msa.msa_shard_lengths(
            z(1, dtype=torch.int32), batch=1, max_kv=64, token_base=0, token_count=32, **kw), 1),
        "shard_lengths_none": (lambda **kw: msa.msa_shard_lengths(
            None, batch=1, max_kv=64, token_base=0, token_count=32, device="cpu", **kw), 1),
        "forward": (lambda **kw: msa.msa_forward(q, k, k, qi, ki, return_ids=True,
                                                 return_scores=True, return_lse=True, **sel, **kw), 4),
    }


@pytest.mark.parametrize("name", sorted(bf16_calls()))
def test_results_of_the_bf16_calls_are_made_on_their_stream(name, streams, monkeypatch):
    side, log = streams
    call, made = bf16_calls()[name]
    buffer = torch.zeros(1 << 16, dtype=torch.uint8)
    empty, empty_like = torch.empty, torch.empty_like

    class Library:
        def __getattr__(self, entry):
            def launch(*args):
                log.append((entry, Recording.current))
                return 0
            return launch

    class Space:
        def get(self, nbytes):
            log.append(("workspace", Recording.current))
            return buffer

    monkeypatch.setattr(msa, "load_library", lambda: Library())
    monkeypatch.setattr(msa, "msa_workspace_size", lambda *a: 4096)
    monkeypatch.setattr(msa, "_workspace", lambda *a: Space())
    monkeypatch.setattr(msa, "_stream", lambda stream=None: stream.cuda_stream if stream else 0)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: (log.append(("empty", Recording.current)),
                                                         empty(*a, **k))[1])
    monkeypatch.setattr(torch, "empty_like", lambda *a, **k: (
        log.append(("empty", Recording.current)), empty_like(*a, **k))[1])
    call(stream=side)
    assert [n for n, _ in log].count("empty") == made and log[-1][0].startswith("msa_")
    assert all(s is side for _, s in log), log
    log.clear()
    call()
    assert all(s is None for _, s in log) and log[-1][0].startswith("msa_")
    if name != "shard_lengths_none":
        side.device.index = 3
        with pytest.raises(ValueError, match="stream"):
            call(stream=side)


# ------------------------------------------------------------------------ on a GPU
def queue_work(ms=10):
    """Milliseconds of work on the current stream."""
    a = torch.randn((4096, 4096), device="cuda").to(BF16)
    for _ in range(ms * 8):  # about 0.1 ms each
        a = torch.mm(a, a)


def filled_cache():
    g = torch.Generator(device="cuda").manual_seed(7)
    c = msa.q8_cache(batch=2, max_kv=1000, h=4, d=128, d_idx=64, block=64)

    def draw(*shape):
        return torch.randn(shape, device="cuda", generator=g).to(BF16)

    msa.msa_append_kv_q8(*c, draw(2, 1000, 4, 128), draw(2, 1000, 4, 128), draw(2, 1000, 64),
                         block=64)
    return c, draw(2, 1, 32, 128), draw(2, 1, 4, 64)


@pytest.mark.gpu
def test_read_on_a_side_stream_while_the_current_one_is_busy():
    c, _, _ = filled_cache()
    want = msa.msa_read_kv_q8(*c, n=900, token_base=50, block=64)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    queue_work()
    got = msa.msa_read_kv_q8(*c, n=900, token_base=50, block=64, stream=side)
    side.synchronize()
    early = [t.clone() for t in got]
    torch.cuda.synchronize()
    for a, b, e in zip(got, want, early):
        assert torch.equal(a, b) and torch.equal(e, b) and bool(a.any())


@pytest.mark.gpu
def test_results_of_a_side_stream_do_not_take_memory_of_the_busy_current_one():
    """Memory that was freed while the current stream still has a write to it queued."""
    c, q, qi = filled_cache()
    kw = dict(block=64, topk=4, return_ids=True, return_scores=True, return_lse=True)
    cache = c.k, c.v, qi, c.k_idx, c.k_scale, c.v_scale, c.k_idx_scale
    want = msa.msa_forward_q8(q, *cache, **kw)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    queue_work()
    held = [torch.full_like(t, 3) for t in want for _ in range(4)]  # queued behind the work
    where = {t.data_ptr() for t in held}
    del held
    got = msa.msa_forward_q8(q, *cache, stream=side, **kw)
    assert not where & {t.data_ptr() for t in got}
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_bf16_results_of_a_side_stream_while_the_current_one_is_busy():
    """With a workspace of its own that this call makes and clears: the clearing is ordered
    before the call, not behind the work of the current stream."""
    c, q, qi = filled_cache()
    k, v, ki = msa.msa_read_kv_q8(*c, n=1000, block=64)
    kw = dict(block=64, topk=8, return_ids=True, return_scores=True, return_lse=True)
    want = msa.msa_forward(q, k, v, qi, ki, **kw)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    queue_work()
    held = [torch.full_like(t, 3) for t in want for _ in range(4)]  # queued behind the work
    where = {t.data_ptr() for t in held}
    del held
    got = msa.msa_forward(q, k, v, qi, ki, workspace=msa.Workspace("cuda"), stream=side, **kw)
    assert not where & {t.data_ptr() for t in got}
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
