"""What each row of ress_masked_attn loses to rounding: no more than its own scores account for.

The tolerances of test_masked_attn.py take the largest distance and score of the whole call.
Here they are each row's own, so that a row's error may not depend on where other queries
and hidden keys lie.  With S = 64 * 2^-23 of the row's largest sum |q k| scale (the products),
D the bias of the row's keys that carry weight (2^-40 of the largest, the others vanish) and
R the row's largest |score|, in units of 2^-24:
  bias    slope log2 e 2 D; a distance is a sum of two terms of one sign, each converted and
          multiplied (2 D); the score added to one (R + D), the other less the maximum
          (D + |max|), and their sum (R + D + |max|), with |max| <= R + D; the key's term may be
          a running sum of up to 15 additions of one sign, the k-th rounding k/15 of it (8 D)
          -> 17 D + 4 R
  cap     tanh within 2^-21 of its value, products and scales 4 roundings -> 12 R
"""
import math

import pytest
import torch

from block_sparse_global_b200 import build as B
from block_sparse_global_b200 import ress as R
from oracle import token_oracle as T

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return R.load()


def _run(q, k, v, key_block=128, scale=0.125, **mods):
    Bn, H, Nq, _ = q.shape
    shape = R.make_shape(Bn, H, k.shape[2], key_block=key_block)
    ws = torch.empty(max(16, R.ress_masked_attn_workspace_bytes(shape, Nq)), dtype=torch.uint8, device="cuda")
    out = torch.full((Bn, H, Nq, 64), 3.0, dtype=BF16, device="cuda")
    lse = torch.full((Bn, H, Nq), 3.0, device="cuda")
    R.ress_masked_attn(shape, q, k, v, None, None, None, scale, out, lse, workspace=ws.fill_(255), **mods)
    return out, lse


def _check_rows(q, k, v, out, lse, scale=0.125, softcap=0.0, slopes=None, q_pos=None, k_pos=None, **masks):
    """Each row against 64 bits by its own tolerance."""
    mods = dict(softcap=softcap, slopes=slopes, q_pos=q_pos, k_pos=k_pos, **masks)
    want, want_lse, size, reach = T.masked_attn(q, k, v, scale, **mods)
    Bn, H, Nq, _ = q.shape
    N = k.shape[2]
    far = torch.zeros_like(reach)
    for b in range(Bn):
        seen = torch.ones(Nq, N, dtype=torch.bool, device=q.device)
        if "q_doc" in masks:
            seen &= (masks["q_doc"][b][:, None] == masks["k_doc"][b]) & (masks["q_doc"][b][:, None] >= 0)
        if "q_order" in masks:
            seen &= masks["k_order"][b] <= masks["q_order"][b][:, None]
        for h in range(H):
            kk = torch.where(seen.any(0)[:, None], k[b, h].double(), torch.zeros((), dtype=torch.float64).cuda())
            s = q[b, h].double() @ kk.T * scale
            if softcap:
                s = softcap * torch.tanh(s / softcap)
            if slopes is None:
                continue
            d = slopes[h].double() * (q_pos[b].double()[:, None] - k_pos[b].double()).abs()
            s = torch.where(seen, s - d, torch.full_like(s, -math.inf))
            near = s >= s.amax(-1, keepdim=True) - 40 * math.log(2)
            far[b, h] = torch.where(near & seen, d.abs(), torch.zeros_like(d)).amax(-1)
    top = reach if not softcap else reach.clamp_max(softcap)
    e = 64 * 2.0 ** -23 * reach + (17 * far + (16 if softcap else 4) * top) * 2.0 ** -24
    none = want_lse == -math.inf
    assert bool((lse[none] == -math.inf).all()) and bool((out[none] == 0).all())
    # exponentials 2^-21, sums a tree a tile, the logarithm's and its own rounding
    tol = e + 2.0 ** -20 + (N / 128 + 8) * 2.0 ** -23 + 2.0 ** -22 * want_lse.abs()
    err = (lse.double() - want_lse).abs()
    assert bool((err[~none] <= tol[~none]).all()), f"lse: worst {float((err / tol)[~none].max()):.2f} of the tolerance"
    tol = (2.0 ** -8 + 2 * e + (N + 64) * 2.0 ** -23).unsqueeze(-1) * size + 2.0 ** -8 * want.abs() + 1e-30
    err = (out.double() - want).abs()
    assert bool((err <= tol).all()), f"out: worst {float((err / tol).max()):.2f} of the tolerance"


def _inputs(H, N, Nq, seed, size=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    mk = lambda n: (size * torch.randn(1, H, n, 64, device="cuda", generator=g)).to(BF16)  # noqa: E731
    return mk(Nq), mk(N), mk(N)


@pytest.mark.gpu
@pytest.mark.parametrize("kb", [64, 128])
@pytest.mark.parametrize("cap", [0.0, 25.0])
def test_queries_of_a_block_far_from_one_another(cap, kb):
    """Positions that restart inside a query block (packed documents, streams): the distance
    is between a query and its keys, however far the block's first query is.  Every path: keys
    behind and ahead of a warp's queries, and warps whose queries lie on both sides."""
    gen = torch.Generator().manual_seed(5)
    bases = [-16000000, 15500001, 3, 5000001, 15999997]
    some = lambda n: torch.randint(0, 230, (n,), generator=gen)  # noqa: E731
    k_pos = torch.cat([x for b in bases for x in (b - some(128), b + 32 + some(128))] + [3 - some(37)])
    rows = torch.arange(32)
    block = torch.cat([bases[0] + rows, bases[1] + rows, bases[2] + rows,
                       torch.where(rows % 2 == 0, bases[3] + rows, bases[4] + rows)])
    q_pos = torch.cat([block, block[torch.randperm(128, generator=gen)]])
    N, Nq = len(k_pos), len(q_pos)
    q, k, v = _inputs(3, N, Nq, seed=3)
    mods = dict(softcap=cap, slopes=torch.tensor([0.5, 1.0, 0.01], device="cuda"),
                q_pos=q_pos.to(torch.int32).view(1, Nq).cuda(), k_pos=k_pos.to(torch.int32).view(1, N).cuda())
    out, lse = _run(q, k, v, kb, **mods)
    _check_rows(q, k, v, out, lse, **mods)


@pytest.mark.gpu
@pytest.mark.parametrize("kb", [64, 128])
@pytest.mark.parametrize("side", [1, -1])
@pytest.mark.parametrize("step", [1, 7, -1000, 40000, -40000])
def test_evenly_spaced_positions_of_any_step(step, side, kb):
    """Keys whose even steps are large, as time stamps are, and queries just behind or ahead of
    them: the key next to a query is not rounded at the magnitude of its block's first one.
    Two whole runs of the same positions and a short one."""
    N, Nq, H = 300, 2000, 3
    q, k, v = _inputs(H, N, Nq, seed=9)
    k_pos = step * (torch.arange(N) % 128)
    q_pos = (k_pos.max() if side > 0 else k_pos.min()) + side * (1 + torch.arange(Nq) % 3)
    mods = dict(slopes=torch.tensor([0.5, 1.0, 0.01], device="cuda"),
                q_pos=q_pos.to(torch.int32).view(1, Nq).cuda(), k_pos=k_pos.to(torch.int32).view(1, N).cuda())
    out, lse = _run(q, k, v, kb, **mods)
    _check_rows(q, k, v, out, lse, **mods)


@pytest.mark.gpu
@pytest.mark.parametrize("kb", [64, 128])
@pytest.mark.parametrize("bias", [0.0, 0.1])
@pytest.mark.parametrize("cap", [0.3, 10.0, 1e4, 1e5])
def test_the_caps_error_is_each_scores_own(cap, bias, kb):
    """Small scores beside ones far above the cap, in one tile: each within its own rounding of
    the cap, which is the identity to the small ones."""
    N, H = 500, 2
    q, k, v = _inputs(H, N, N, seed=22)
    q[:, :, 5::32] *= 1000 * max(1.0, cap)   # a row of every warp
    k[:, :, 7::128] *= 30                    # and a key of every tile
    mods = dict(softcap=cap)
    if bias:
        t = torch.arange(N, dtype=torch.int32, device="cuda").view(1, N)
        mods.update(slopes=torch.full((H,), bias, device="cuda"), q_pos=t, k_pos=t)
    out, lse = _run(q, k, v, kb, **mods)
    _check_rows(q, k, v, out, lse, **mods)


@pytest.mark.gpu
@pytest.mark.parametrize("kb", [64, 128])
@pytest.mark.parametrize("cap", [2.0, 30.0, 1e4])
@pytest.mark.parametrize("bias", [0.0, 0.1])
@pytest.mark.parametrize("hidden", [float("inf"), float("nan"), 1e4])
def test_capped_rows_do_not_change_with_keys_that_they_do_not_see(hidden, bias, cap, kb):
    """A later key, whatever it holds, leaves every bit of the rows before it, although rows of
    the same warp see it; so does a key that no query sees."""
    N, H = 400, 4                            # (the form for few rows takes less)
    q, k, v = _inputs(H, N, N, seed=21)
    t = torch.arange(N, dtype=torch.int32, device="cuda").view(1, N)
    doc = (t >= 390).to(torch.int32) * -1
    mods = dict(softcap=cap, q_order=t, k_order=t, q_doc=doc, k_doc=doc)
    if bias:
        mods.update(slopes=torch.full((H,), bias, device="cuda"), q_pos=t, k_pos=t)
    clean, lse = _run(q, k, v, kb, **mods)
    _check_rows(q, k, v, clean, lse, **mods)
    k2, v2 = k.clone(), v.clone()
    k2[:, :, 300, 0] = hidden                # rows 288 to 299 share a warp with those that see it
    k2[:, :, 395, 0] = hidden                # padding
    v2[:, :, 300, 3] = hidden
    out, lse2 = _run(q, k2, v2, kb, **mods)
    assert torch.equal(out[:, :, :300], clean[:, :, :300]) and torch.equal(lse2[:, :, :300], lse[:, :, :300])
    assert not torch.equal(out[:, :, 300:], clean[:, :, 300:])


@pytest.mark.gpu
@pytest.mark.parametrize("scale,cap", [(1e10, 1.01e5), (1e30, 1.01e25), (3e-36, 4e-36), (1e-38, 1e-34), (0.125, 50.0)])
def test_scales_and_caps_at_the_ends_of_their_ranges(scale, cap):
    """Zero queries see every key alike, whatever the scale: the mean of the values."""
    H, N = 4, 700
    q, k, v = _inputs(H, N, N, seed=23)
    out, lse = _run(q * 0, k, v, scale=scale, softcap=cap)
    mean = v.double().mean(2, keepdim=True)
    size = v.double().abs().mean(2, keepdim=True)
    # the weights are exactly 1; sums of N values, the sum's reciprocal and the output's rounding
    assert bool(((out.double() - mean).abs() <= 2.0 ** -8 * mean.abs() + (N + 64) * 2.0 ** -23 * size).all())
    assert float((lse.double() - math.log(N)).abs().max()) <= 2.0 ** -20 + 2.0 ** -22 * math.log(N)
