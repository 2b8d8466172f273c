"""The workspace of ress_masked_attn: none where the form for few rows takes the call."""
import pytest
import torch

from block_sparse_global_b200 import build as B
from block_sparse_global_b200 import ress as R
from block_sparse_global_b200.pipeline import SparseGlobalAttention

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return R.load()


def test_few_rows_need_none():
    for heads, tokens, queries in ((16, 10992, 1), (4, 700, 3), (1, 1, 1), (128, 10992, 1)):
        assert R.ress_masked_attn_workspace_bytes(R.make_shape(1, heads, tokens), queries) == 0
    for heads, tokens, queries in ((16, 10992, 128), (16, 43968, 1), (4, 1024, 1024)):
        assert R.ress_masked_attn_workspace_bytes(R.make_shape(1, heads, tokens), queries) > 0


def test_a_layer_keeps_none_for_few_rows(monkeypatch):
    layer = SparseGlobalAttention(1, 4, 3000, device="cpu")
    seen = []
    monkeypatch.setattr(R, "ress_masked_attn", lambda *a, workspace=None, **kw: seen.append(workspace))
    k = torch.zeros(1, 4, 3000, 64, dtype=BF16)
    for n in (1, 2, 100, 1, 128):                      # the last three in one query block
        layer.attend_masked(torch.zeros(1, 4, n, 64, dtype=BF16), k, k, kept=False)
    sizes = [0 if w is None else w.numel() for w in seen]
    assert sizes[0] == sizes[1] == sizes[3] == 0 and seen[2] is seen[4]
    for n in (100, 101, 128):
        assert sizes[2] == R.ress_masked_attn_workspace_bytes(layer.shape, n)


@pytest.mark.gpu
def test_a_call_without_one():
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn(1, 4, n, 64, device="cuda", generator=g).to(BF16) for n in (2, 900, 900))
    shape, outs = R.make_shape(1, 4, 900), []
    for ws in (None, torch.empty(0, dtype=torch.uint8, device="cuda"),
               torch.empty(64, dtype=torch.uint8, device="cuda")):
        outs.append(torch.empty_like(q))
        R.ress_masked_attn(shape, q, k, v, None, None, None, 0.125, outs[-1], workspace=ws)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    s = torch.softmax(q.double() @ k.double().transpose(2, 3) * 0.125, -1)
    assert float((outs[0].double() - s @ v.double()).abs().max()) <= 2.0 ** -8 * 4
    with pytest.raises(R.RessError):                   # 600 queries: tensor-core tiles, summaries
        big = torch.zeros(1, 4, 600, 64, dtype=BF16, device="cuda")
        R.ress_masked_attn(shape, big, k, v, None, None, None, 0.125, torch.empty_like(big))
