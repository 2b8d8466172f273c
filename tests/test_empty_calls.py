"""Empty problems: an array without elements has no address, and is not asked for one."""
import ctypes
import math

import pytest
import torch

from block_sparse_global_b200 import build as B
from block_sparse_global_b200 import ress as R

BF16, I32 = torch.bfloat16, torch.int32
FAKE = 0x7F0000000000
OK, INVALID = 0, 1


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return R.load()


def test_token_operators_without_tokens(lib):
    plan = R.rope_plan(64, axes=2)                     # two axes: positions are needed
    rows = ctypes.byref(R.ress_rows(None, 0, 64, 128))

    def rope(tokens, batch=1):
        return lib.ress_rope(ctypes.byref(plan), batch, 2, tokens, 0, rows, None, 0, 0, rows, None)

    def qk(tokens, batch=1):
        p = R.ress_qk_params(batch, tokens, 2, 2, 64, 0, 1, 1e-6, None, None, None, None, ctypes.addressof(plan),
                             None, 0, 1, 0)
        return lib.ress_qk_norm_rope(ctypes.byref(p), rows, rows, None, rows, rows, None, None)

    for call in (rope, qk):
        assert call(0) == OK and call(5, batch=0) == OK
        assert call(5) == INVALID


def test_masked_attention_without_queries(lib):
    def call(q_len, **arrays):
        m = R.ress_attn_mods(q_len)
        for n, x in arrays.items():
            if n != "cnt":
                setattr(m, n, x)
        return lib.ress_masked_attn(ctypes.byref(R.make_shape(1, 2, 1000)), ctypes.byref(m), None, FAKE, FAKE, None,
                                    arrays.get("cnt"), None, 0.125, None, None, None, 0, None, None)

    for arrays in (dict(k_doc=FAKE), dict(k_order=FAKE), dict(k_pos=FAKE, slopes=FAKE), dict(cnt=FAKE)):
        assert call(0, **arrays) == OK
        assert call(5, **arrays) == INVALID


@pytest.mark.gpu
@pytest.mark.parametrize("lists", [False, True])
def test_masked_attention_without_keys(lists):
    """Every query has a zero row, with masks, a bias and lists as without."""
    H, Nq = 2, 130
    q = torch.randn(1, H, Nq, 64, device="cuda").to(BF16)
    k = torch.empty(1, H, 0, 64, device="cuda", dtype=BF16)
    row, none = torch.zeros(1, Nq, dtype=I32, device="cuda"), torch.empty(1, 0, dtype=I32, device="cuda")
    idx = torch.empty(1, H, 2, 0, dtype=I32, device="cuda") if lists else None
    cnt = torch.zeros(1, H, 2, dtype=I32, device="cuda") if lists else None
    out = torch.full_like(q, 3.0)
    lse = torch.full((1, H, Nq), 3.0, device="cuda")
    R.ress_masked_attn(R.make_shape(1, H, 0), q, k, k, idx, cnt, None, 0.125, out, lse, q_doc=row, k_doc=none,
                       q_order=row, k_order=none, q_pos=row, k_pos=none, slopes=torch.ones(H, device="cuda"))
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


@pytest.mark.gpu
def test_empty_tensors_through_the_bindings():
    x = torch.empty(2, 3, 0, 64, device="cuda", dtype=BF16)
    pos = torch.empty(2, 0, 2, device="cuda", dtype=I32)
    plan = R.rope_plan(64, axes=2)
    R.ress_rope(plan, x, pos, torch.empty_like(x))
    R.ress_qk_norm_rope(x, x, torch.empty_like(x), torch.empty_like(x), plan=plan, positions=pos)
    k = torch.randn(2, 3, 40, 64, device="cuda").to(BF16)
    row, none = torch.zeros(2, 40, dtype=I32, device="cuda"), torch.empty(2, 0, dtype=I32, device="cuda")
    R.ress_masked_attn(R.make_shape(2, 3, 40), x, k, k, None, None, None, 0.125, torch.empty_like(x), q_order=none,
                       k_order=row)
    torch.cuda.synchronize()
