"""Which stream the layer's own buffers belong to.

The caching allocator may hand out memory whose last kernel on the allocating stream still
runs; only that stream is ordered behind it.  What a call makes for itself must therefore be
made on the stream that the call runs on.
"""
import contextlib
import types

import pytest
import torch

from block_sparse_global_b200 import build as B
from block_sparse_global_b200 import pipeline as P
from block_sparse_global_b200 import ress as R

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()


# ------------------------------------------------------------------------ on the host
class FakeStream:
    def __init__(self, number):
        self.cuda_stream = number


@pytest.fixture
def fake(monkeypatch):
    """CUDA's streams faked on the CPU: the stream that is current where a tensor is made, and
    the streams that tensors are said to be used on."""
    seen = types.SimpleNamespace(now=FakeStream(0), made={}, used={}, calls=[])
    real_empty = torch.empty

    @contextlib.contextmanager
    def stream(s):
        before, seen.now = seen.now, s
        yield
        seen.now = before

    def empty(*a, **kw):
        t = real_empty(*a, **kw)
        seen.made[t.data_ptr()] = seen.now.cuda_stream
        return t

    def note(name):
        def call(*a, stream=None, **kw):
            seen.calls.append((name, seen.now.cuda_stream if stream is None else stream.cuda_stream, a, kw))
        return call

    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda n, device=None: FakeStream(n))
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: seen.now)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, s: seen.used.setdefault(t.data_ptr(), set()).add(s.cuda_stream))
    monkeypatch.setattr(R, "ress_masked_attn", note("attn"))
    monkeypatch.setattr(R, "ress_qk_norm_rope", note("qk"))
    return seen


def test_default_output_and_workspace_are_made_on_the_calls_stream(fake):
    layer = P.SparseGlobalAttention(1, 2, 3000, device="cpu")
    k = torch.zeros(1, 2, 3000, 64, dtype=BF16)
    q = torch.zeros(1, 2, 1500, 64, dtype=BF16)
    out = layer.attend_masked(q, k, k, kept=False, stream=FakeStream(7))
    ws = fake.calls[-1][3]["workspace"]
    assert fake.made[out.data_ptr()] == 7 and fake.made[ws.data_ptr()] == 7
    assert 0 in fake.used[out.data_ptr()]          # the caller reads it on the current stream
    out = layer.attend_masked(q, k, k, kept=False)
    assert fake.made[out.data_ptr()] == 0 and out.data_ptr() not in fake.used


def test_prepared_tensors_are_made_on_the_calls_stream(fake):
    layer = P.SparseGlobalAttention(1, 2, 300, device="cpu")
    packed = torch.zeros(1, 300, 3, 2, 64, dtype=BF16)
    for t in layer.prepare(packed, stream=FakeStream(9)):
        assert fake.made[t.data_ptr()] == 9 and 0 in fake.used[t.data_ptr()]


def test_projection_is_converted_on_the_calls_stream(fake, monkeypatch):
    layer = P.SparseGlobalAttention(1, 2, 300, device="cpu")
    real, where = torch.Tensor.float, []
    monkeypatch.setattr(torch.Tensor, "float", lambda t: where.append(fake.now.cuda_stream) or real(t))
    monkeypatch.setattr(R, "ress_head_gram", lambda *a: None)
    layer.load_output_projection(torch.zeros(128, 128, dtype=BF16), stream=FakeStream(5))
    layer.load_output_projection(torch.zeros(128, 128, dtype=BF16))
    assert where == [5, 0]


def test_a_refused_call_leaves_no_buffer_behind(fake, monkeypatch):
    """A buffer of a call that never ran would belong to a stream that nothing is ordered by."""
    layer = P.SparseGlobalAttention(1, 2, 3000, device="cpu")
    q = torch.zeros(1, 2, 1500, 64, dtype=BF16)

    def refuse(*a, **kw):
        raise ValueError

    ran = R.ress_masked_attn, R.ress_qk_norm_rope
    monkeypatch.setattr(R, "ress_masked_attn", refuse)
    monkeypatch.setattr(R, "ress_qk_norm_rope", refuse)
    packed = torch.zeros(1, 3000, 3, 2, 64, dtype=BF16)
    with pytest.raises(ValueError):
        layer.attend_masked(q, q, q, kept=False, stream=FakeStream(7))
    with pytest.raises(ValueError):
        layer.prepare(packed, stream=FakeStream(7))
    monkeypatch.setattr(R, "ress_masked_attn", ran[0])
    monkeypatch.setattr(R, "ress_qk_norm_rope", ran[1])
    layer.attend_masked(q, q, q, kept=False, stream=FakeStream(8))
    assert fake.made[fake.calls[-1][3]["workspace"].data_ptr()] == 8
    assert all(fake.made[t.data_ptr()] == 8 for t in layer.prepare(packed, stream=FakeStream(8)))


# ------------------------------------------------------------------------- on the GPU
def _busy(nbytes):
    """Work on the current stream whose freed buffer the allocator would hand out next: a chain
    of products of some milliseconds, then a fill of nbytes bytes."""
    a = torch.randn(4096, 4096, device="cuda").to(BF16)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    junk = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    for _ in range(30):
        a = a @ a * 1e-3
    junk.fill_(77)
    return a


@pytest.mark.gpu
@pytest.mark.parametrize("as_handle", [False, True])
def test_new_tokens_on_a_side_stream_beside_a_busy_one(as_handle):
    g = torch.Generator(device="cuda").manual_seed(1)
    N, n, H = 9000, 300, 3
    layer = P.SparseGlobalAttention(1, H, N)
    q, k, v = (torch.randn(1, H, m, 64, device="cuda", generator=g).to(BF16) for m in (n, N, N))
    want = P.SparseGlobalAttention(1, H, N).attend_masked(q, k, v, kept=False, softcap=9.0)
    size = R.ress_masked_attn_workspace_bytes(layer.shape, n)
    side = torch.cuda.Stream()
    handle = side.cuda_stream if as_handle else side
    torch.cuda.synchronize()
    for nbytes in (size, H * n * 64 * 2):
        keep = _busy(nbytes)
        out = layer.attend_masked(q, k, v, kept=False, softcap=9.0, stream=handle)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and keep.shape == (4096, 4096)


@pytest.mark.gpu
def test_prepare_on_a_side_stream_beside_a_busy_one():
    g = torch.Generator(device="cuda").manual_seed(2)
    N, H = 4000, 4
    packed = torch.randn(1, N, 3, H, 64, device="cuda", generator=g).to(BF16)
    plan = R.rope_plan(64)
    want = [t.clone() for t in P.SparseGlobalAttention(1, H, N).prepare(packed, plan, norm=R.NORM_RMS)]
    layer = P.SparseGlobalAttention(1, H, N)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    keep = _busy(H * N * 64 * 2)
    got = layer.prepare(packed, plan, norm=R.NORM_RMS, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and keep.shape == (4096, 4096)
