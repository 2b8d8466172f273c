"""Rotary positions and the per-head norm (ress_rope, ress_qk_norm_rope) against 64 bits.

Tolerances, u = 2^-24 (half an fp32 step), per element:
  rope   the angle left after whole quarter turns is at most pi/4 and rounded once (0.8 u),
         sincospi is within 2 steps (4 u), the amplitude's product, the product of a term and
         the fused sum round once each (3 u): 8 u A (|x_a| + |x_b|), plus the rounding to the
         stored type.
  norm   a sum of at most 256 terms in lanes and shuffles passes at most 8 + 8 + 5 roundings,
         half of which reach 1/sqrt; with the division, rsqrt (2 steps), the mean's own error
         (as large, against the row's largest element), the affine map and the rounding of
         the centred element, less than 40 u (max|x| r max|w| + max|b|) per element; the
         rotation then carries at most twice that.
"""
import ctypes

import pytest
import torch

from block_sparse_global_b200 import build as B
from block_sparse_global_b200 import ress as R
from block_sparse_global_b200 import workload as W
from block_sparse_global_b200.pipeline import SparseGlobalAttention
from oracle import token_oracle as T

INVALID, UNSUPPORTED, OK = 1, 2, 0
FAKE = 0x7F0000000000
U = 2.0 ** -24
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return R.load()


# ------------------------------------------------------------------------ on the host
@pytest.mark.parametrize("scaling,kw", [("none", {}), ("linear", dict(factor=4.0)), ("ntk", dict(factor=8.0)),
                                        ("yarn", dict(factor=8.0, original_len=4096)),
                                        ("yarn", dict(factor=40.0, original_len=3))])
@pytest.mark.parametrize("head_dim,rot,axes", [(64, 64, 1), (96, 36, 3), (256, 256, 1), (80, 8, 2)])
def test_plan_holds_the_frequencies(scaling, kw, head_dim, rot, axes):
    plan = R.rope_plan(head_dim, rot, axes=axes, theta=10000.0, scaling=scaling, **kw)
    f, amp = T.frequencies(rot // axes, 10000.0, scaling, **kw)
    assert plan.amplitude == pytest.approx(amp, rel=2 * U)
    for i, w in enumerate(f):
        # turns per position: the plan rounds at 2^-65, the double formula at 2^-50 relative
        assert plan.phase[i] * 2.0 ** -64 == pytest.approx(w / 6.283185307179586, rel=1e-14, abs=2.0 ** -64)


@pytest.mark.parametrize("bad", [
    dict(head_dim=0), dict(head_dim=257), dict(rot_dim=0), dict(rot_dim=66), dict(rot_dim=7), dict(axes=0),
    dict(axes=4), dict(axes=3), dict(theta=1.0), dict(theta=float("nan")), dict(theta=1e13),
    dict(scaling="linear", factor=0.5), dict(scaling="linear", factor=float("inf")),
    dict(scaling="ntk", factor=2.0, rot_dim=2), dict(scaling="yarn", factor=2.0, original_len=0),
    dict(scaling="yarn", factor=2.0, original_len=64, beta_slow=0.0),
    dict(scaling="yarn", factor=2.0, original_len=64, beta_slow=32.0)])
def test_plan_refusals(bad):
    kw = dict(head_dim=64)
    kw.update(bad)
    with pytest.raises(R.RessError) as e:
        R.rope_plan(**kw)
    assert e.value.status == INVALID


def test_plan_names():
    with pytest.raises(ValueError):
        R.rope_plan(64, layout="other")
    with pytest.raises(ValueError):
        R.rope_plan(64, scaling="other")


def _view(ptr=FAKE, b=0, h=64, t=128):
    return ctypes.byref(R.ress_rows(ptr, b, h, t))


def test_rope_refusals(lib):
    plan = R.rope_plan(64)

    def call(plan=plan, B=1, H=2, N=5, dtype=0, x=None, pos=None, pos_b=0, inv=0, out=None):
        x = _view() if x is None else x
        out = _view(FAKE + 65536) if out is None else out
        return lib.ress_rope(ctypes.byref(plan) if plan else None, B, H, N, dtype, x, pos, pos_b, inv, out, None)

    assert call(plan=None) == INVALID
    assert call(B=-1) == INVALID and call(H=-1) == INVALID and call(N=-1) == INVALID
    assert call(dtype=3) == INVALID and call(dtype=-1) == INVALID
    assert call(inv=2) == INVALID
    assert call(pos=FAKE + 2) == INVALID and call(pos=FAKE, pos_b=-1) == INVALID
    assert call(x=_view(None)) == INVALID and call(out=_view(None)) == INVALID
    assert call(x=_view(FAKE + 1)) == INVALID                        # half an element
    assert call(x=_view(t=-128)) == INVALID
    assert call(out=_view(FAKE + 65536, h=0)) == INVALID             # rows on top of one another
    assert call(out=_view(FAKE + 65536, h=32)) == INVALID
    assert call(out=_view(FAKE + 65536, t=64)) == INVALID            # h and t share rows
    assert call(out=_view(t=256)) == INVALID                         # in place, other strides
    assert call(plan=R.rope_plan(64, axes=2), pos=None) == INVALID   # axes need positions
    bad = R.rope_plan(64)
    bad.rot_dim = 65
    assert call(plan=bad) == INVALID
    bad = R.rope_plan(64)
    bad.amplitude = 0.0
    assert call(plan=bad) == INVALID
    assert call(H=65537, out=_view(FAKE + 65536, t=64 * 65537)) == UNSUPPORTED
    assert call(N=0, x=_view(None), out=_view(None)) == OK           # empty: nothing is looked at
    assert call(B=0) == OK and call(H=0) == OK


def test_qk_refusals(lib):
    plan = R.rope_plan(64)

    def call(v=None, v_out=None, q=None, q_out=None, k_out=None, **kw):
        p = R.ress_qk_params(1, 10, 2, 2, 64, 0, 1, 1e-6, None, None, None, None, ctypes.addressof(plan), None, 0,
                             1, 0)
        for n, x in kw.items():
            setattr(p, n, x)
        return lib.ress_qk_norm_rope(ctypes.byref(p), q or _view(), _view(FAKE + 4096), v,
                                     q_out or _view(FAKE + 65536), k_out or _view(FAKE + 2 * 65536), v_out, None)

    assert lib.ress_qk_norm_rope(None, *([_view()] * 6), None) == INVALID
    for bad in (dict(batch=-1), dict(tokens=-1), dict(q_heads=0), dict(kv_heads=0), dict(head_dim=1),
                dict(head_dim=258), dict(head_dim=128), dict(dtype=5), dict(norm=3), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(q_weight=FAKE + 2), dict(views=0),
                dict(views=3), dict(specials=-1), dict(views=2, specials=6), dict(positions=FAKE + 1),
                dict(v=_view(FAKE + 8192)), dict(v_out=_view(FAKE + 8192)),
                dict(q_out=_view(FAKE + 65536, h=0)), dict(k_out=_view(FAKE + 65536)), dict(k_out=_view())):
        assert call(**bad) == INVALID, bad
    # in place is for calls that keep the token order, and for equal strides
    assert call(q_out=_view(), specials=2) == INVALID
    assert call(q_out=_view(h=1280, t=64)) == INVALID
    assert call(q_heads=65537) == UNSUPPORTED and call(kv_heads=65537) == UNSUPPORTED
    assert call(batch=0) == OK and call(tokens=0) == OK


def test_binding_refuses_what_does_not_fit():
    plan = R.rope_plan(64)
    x = torch.zeros(1, 2, 5, 64, dtype=BF16)
    with pytest.raises(ValueError):
        R.ress_rope(plan, x, None, torch.zeros(1, 2, 4, 64, dtype=BF16))       # another shape
    with pytest.raises(ValueError):
        R.ress_rope(plan, x, None, torch.zeros(1, 2, 5, 64))                    # another type
    with pytest.raises(ValueError):
        R.ress_rope(plan, x.double(), None, x.double())
    with pytest.raises(ValueError):
        R.ress_rope(R.rope_plan(32), x, None, torch.empty_like(x))
    with pytest.raises(ValueError):
        R.ress_rope(plan, x.transpose(2, 3).contiguous().transpose(2, 3), None, torch.empty_like(x))
    for p in (torch.zeros(1, 4), torch.zeros(5, dtype=torch.int64), torch.zeros(4, dtype=torch.int32),
              torch.zeros(2, 5, dtype=torch.int32), torch.zeros(1, 5, 2, dtype=torch.int32),
              torch.zeros(10, dtype=torch.int32)[::2]):
        with pytest.raises(ValueError):
            R.ress_rope(plan, x, p, torch.empty_like(x))
    with pytest.raises(ValueError):
        R.ress_rope(plan, x, None, torch.empty_like(x))                         # not on a GPU
    y = torch.empty_like(x)
    with pytest.raises(ValueError):
        R.ress_qk_norm_rope(x, x, y, torch.empty_like(x), v=x)
    with pytest.raises(ValueError):
        R.ress_qk_norm_rope(x, x[:, :, :4], y, torch.empty_like(x))
    with pytest.raises(ValueError):
        R.ress_qk_norm_rope(x, x, y, torch.empty_like(x), q_weight=torch.ones(32))
    with pytest.raises(ValueError):
        R.ress_qk_norm_rope(x, x, y, torch.empty_like(x), q_weight=torch.ones(64, dtype=BF16))


# ------------------------------------------------------------------------- on the GPU
def _step(y, dt):
    """Half a step of the stored type at y, and of its subnormals."""
    fi = torch.finfo(dt)
    return fi.eps / 2 * y.abs() + fi.tiny * fi.eps


def _pair_sizes(x, rot, axes, layout):
    """|x_a| + |x_b| of each element's pair (0 where the element is not rotated)."""
    out = torch.zeros_like(x)
    for e0, e1, _, _ in T.pair_elements(rot, axes, layout):
        m = x[..., e0].abs() + x[..., e1].abs()
        out[..., e0] = m
        out[..., e1] = m
    return out


def _check_rope(x, got, positions, rot, axes, layout, freq, amp, inverse=False):
    xd = x.double()
    want = T.rope(xd, positions, rot, axes, layout, freq, amp, inverse)
    # the frequency itself: the plan's 2^-65 turns and the oracle's double product, per position
    far = positions.double().abs().amax(-1)[:, None, :, None] * 2.0 ** -52
    size = _pair_sizes(xd, rot, axes, layout)
    tol = _step(want, x.dtype) * (1 + 16 * U) + (8 * U + far) * amp * size
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), f"worst {float((err / tol.clamp_min(1e-300)).max()):.2f} of the tolerance"


ROPE_CASES = [  # dim, rot, axes, layout, dtype, B, H, N
    (64, 64, 1, "half", BF16, 1, 1, 1), (64, 64, 1, "interleaved", FP16, 16, 16, 1),
    (64, 64, 1, "half", FP32, 2, 3, 77), (128, 96, 1, "half", FP32, 2, 8, 129),
    (128, 48, 1, "interleaved", BF16, 3, 5, 63), (96, 36, 3, "half", FP16, 2, 5, 31),
    (96, 96, 3, "interleaved", FP32, 1, 2, 33), (80, 80, 1, "half", BF16, 2, 12, 40),
    (256, 256, 2, "half", FP32, 1, 2, 20), (256, 128, 1, "half", BF16, 1, 3, 65),
    (32, 2, 1, "half", BF16, 1, 7, 19), (64, 10, 1, "interleaved", FP16, 1, 3, 19), (2, 2, 1, "half", FP32, 1, 2, 9),
    (33, 32, 2, "interleaved", BF16, 2, 2, 50), (254, 252, 3, "half", FP16, 1, 1, 8),
    (64, 64, 2, "half", BF16, 1, 2, 20011), (72, 40, 1, "half", FP16, 1, 1, 70001),
    (64, 20, 1, "half", FP32, 2, 3, 33), (64, 36, 1, "half", BF16, 2, 3, 33), (68, 68, 1, "interleaved", FP16, 1, 2, 9),
    (128, 72, 3, "half", FP32, 1, 2, 11)]


@pytest.mark.gpu
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("dim,rot,axes,layout,dt,Bn,H,N", ROPE_CASES)
def test_rope_against_64_bits(dim, rot, axes, layout, dt, Bn, H, N, inverse):
    g = torch.Generator(device="cuda").manual_seed(dim * 7 + rot + N)
    x = torch.randn(Bn, H, N, dim, device="cuda", generator=g).to(dt)
    pos = torch.randint(-70000, 1 << 22, (Bn, N, axes), device="cuda", generator=g, dtype=torch.int32)
    plan = R.rope_plan(dim, rot, axes=axes, layout=layout)
    freq, amp = T.frequencies(rot // axes, 10000.0)
    guard = torch.full((Bn * H * N * dim + 64,), 7.0, device="cuda", dtype=dt)
    out = guard[32:32 + x.numel()].view(x.shape)
    R.ress_rope(plan, x, pos, out, inverse=inverse)
    torch.cuda.synchronize()
    _check_rope(x, out, pos, rot, axes, layout, freq, amp, inverse)
    assert torch.equal(out[..., rot:], x[..., rot:])
    assert bool((guard[:32] == 7).all()) and bool((guard[-32:] == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("scaling,kw", [("linear", dict(factor=4.0)), ("ntk", dict(factor=8.0)),
                                        ("yarn", dict(factor=40.0, original_len=4096))])
def test_rope_scaled_frequencies(scaling, kw):
    x = torch.randn(2, 3, 41, 64, device="cuda")
    pos = torch.randint(0, 200000, (2, 41, 1), device="cuda", dtype=torch.int32)
    plan = R.rope_plan(64, theta=500000.0, scaling=scaling, **kw)
    freq, amp = T.frequencies(64, 500000.0, scaling, **kw)
    out = torch.empty_like(x)
    R.ress_rope(plan, x, pos, out)
    _check_rope(x, out, pos, 64, 1, "half", freq, amp)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_positions_shapes_far_and_absent(layout):
    """Shared, per-batch and absent positions; angles exact at the far end of int32 (against
    integer arithmetic on the plan, since a double product is off there)."""
    x = torch.randn(3, 2, 21, 64, device="cuda")
    plan = R.rope_plan(64, layout=layout)
    freq, amp = T.frequencies(64, 10000.0)
    out = torch.empty_like(x)
    R.ress_rope(plan, x, None, out)
    iota = torch.arange(21, device="cuda", dtype=torch.int32)
    _check_rope(x, out, iota.view(1, 21, 1).expand(3, 21, 1), 64, 1, layout, freq, amp)
    for p in (iota, iota.view(1, 21), iota.view(21, 1), iota.view(1, 21, 1).expand(1, 21, 1)):
        again = torch.empty_like(x)
        R.ress_rope(plan, x, p, again)
        assert torch.equal(again, out)
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345], dtype=torch.int32, device="cuda")
    y = torch.zeros(1, 1, 3, 64, device="cuda")
    first = torch.tensor([e[0] for e in T.pair_elements(64, 1, layout)], device="cuda")
    second = torch.tensor([e[1] for e in T.pair_elements(64, 1, layout)], device="cuda")
    y[..., first] = 1.0
    z = torch.empty_like(y)
    R.ress_rope(plan, y, pos, z)
    for t, p in enumerate(pos.tolist()):
        turn = torch.tensor([((p * plan.phase[i]) % (1 << 64)) / 2.0 ** 64 for i in range(32)], dtype=torch.float64)
        turn = turn * 6.283185307179586
        assert float((z[0, 0, t, first].cpu().double() - torch.cos(turn)).abs().max()) <= 9 * U
        assert float((z[0, 0, t, second].cpu().double() - torch.sin(turn)).abs().max()) <= 9 * U


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF16, FP32])
def test_rope_strides_offsets_and_in_place(dt):
    """Token-major views, rows off the 16-byte boundary, gaps between rows, and in place: the
    same values whatever the layout; gaps and neighbours stay."""
    base = torch.randn(2, 37, 5, 64, device="cuda").to(dt)
    plan = R.rope_plan(64, 48)
    want = torch.empty(2, 5, 37, 64, device="cuda", dtype=dt)
    R.ress_rope(plan, base.transpose(1, 2).contiguous(), None, want)
    out = torch.empty_like(base).transpose(1, 2)
    R.ress_rope(plan, base.transpose(1, 2), None, out)
    assert torch.equal(out, want)
    for off, gap in ((1, 0), (3, 5), (0, 8), (8, 16)):
        wide = torch.full((2, 37, 5, 64 + off + gap), 5.0, device="cuda", dtype=dt)
        view = wide[..., off:off + 64]
        view.copy_(base)
        R.ress_rope(plan, view.transpose(1, 2), None, view.transpose(1, 2))      # in place
        # the element form may contract products and sums otherwise: one step of the type
        ref = want.transpose(1, 2).double()
        assert bool(((view.double() - ref).abs() <= 2 * _step(ref, dt) + 16 * U).all())
        assert bool((wide[..., :off] == 5).all()) and bool((wide[..., off + 64:] == 5).all())
    broad = base[:, :, :1].expand(2, 37, 5, 64).transpose(1, 2)                   # one head for all
    out = torch.empty(2, 5, 37, 64, device="cuda", dtype=dt)
    R.ress_rope(plan, broad, None, out)
    assert torch.equal(out, want[:, :1].expand_as(out))


@pytest.mark.gpu
def test_rope_inverse_undoes_and_is_the_gradient():
    x = torch.randn(2, 3, 50, 64, device="cuda")
    gy = torch.randn_like(x)
    pos = torch.randint(0, 4000, (2, 50), device="cuda", dtype=torch.int32)
    plan = R.rope_plan(64, 32)
    y, back, gx = (torch.empty_like(x) for _ in range(3))
    R.ress_rope(plan, x, pos, y)
    R.ress_rope(plan, y, pos, back, inverse=True)
    assert float((back - x).abs().max()) <= 40 * U * float(x.abs().max())
    R.ress_rope(plan, gy, pos, gx, inverse=True)
    xr = x.double().requires_grad_()
    f, amp = T.frequencies(32, 10000.0)
    T.rope(xr, pos.unsqueeze(-1), 32, 1, "half", f, amp).backward(gy.double())
    assert float((gx.double() - xr.grad).abs().max()) <= 20 * U * float(gy.abs().max()) + 4000 * 2.0 ** -50
    # and against differences of the forward call
    step = 0.25
    for e in (0, 5, 16, 31, 40):
        plus, minus = x.clone(), x.clone()
        plus[..., e] += step
        minus[..., e] -= step
        yp, ym = torch.empty_like(x), torch.empty_like(x)
        R.ress_rope(plan, plus, pos, yp)
        R.ress_rope(plan, minus, pos, ym)
        slope = ((yp.double() - ym.double()) / (2 * step) * gy.double()).sum(-1)
        assert float((slope - gx[..., e].double()).abs().max()) <= 1e-4


QK_CASES = [  # dim, rot, axes, layout, dtype, B, H, G, N, norm, affine, with_v, views, specials
    (64, 64, 1, "half", BF16, 8, 16, 4, 1, "rms", True, True, 1, 0),
    (64, 64, 2, "half", BF16, 1, 16, 16, 4 * 140, "layer", True, True, 4, 5),
    (128, 48, 1, "interleaved", FP16, 3, 12, 6, 57, "rms", True, False, 1, 0),
    (128, 128, 1, "half", FP32, 1, 5, 5, 33, "layer", False, True, 3, 11),
    (96, 48, 3, "half", FP16, 2, 10, 5, 30, "rms", True, True, 2, 3),
    (80, 16, 1, "interleaved", FP32, 2, 2, 1, 17, "layer", True, True, 1, 4),
    (256, 256, 1, "half", FP32, 1, 8, 2, 12, "rms", False, True, 1, 0),
    (256, 64, 1, "half", BF16, 2, 1, 1, 40, "layer", True, True, 4, 1),
    (31, 30, 3, "half", BF16, 1, 3, 1, 21, "layer", True, True, 7, 2),
    (64, 0, 1, "half", BF16, 2, 3, 3, 50, "rms", True, True, 1, 0),
    (64, 64, 1, "half", BF16, 1, 12, 12, 30, "none", False, True, 5, 1),
    (32, 32, 1, "interleaved", FP16, 1, 1, 1, 40011, "rms", True, True, 1, 0),
    (64, 36, 1, "half", BF16, 2, 5, 1, 66, "layer", True, True, 3, 2),
    (72, 24, 3, "half", FP16, 1, 3, 3, 21, "none", False, True, 1, 0),
    (80, 20, 1, "half", FP32, 1, 4, 2, 19, "rms", True, True, 1, 0)]


@pytest.mark.gpu
@pytest.mark.parametrize("dim,rot,axes,layout,dt,Bn,H,G,N,norm,affine,with_v,views,specials", QK_CASES)
def test_qk_against_64_bits(dim, rot, axes, layout, dt, Bn, H, G, N, norm, affine, with_v, views, specials):
    g = torch.Generator(device="cuda").manual_seed(dim + 31 * N + H)
    packed = torch.randn(Bn, N, H + 2 * G, dim, device="cuda", generator=g)
    packed = (packed * (0.1 + 3 * torch.rand(1, 1, H + 2 * G, 1, device="cuda", generator=g)) + 0.5).to(dt)
    keep = packed.clone()
    x = packed.transpose(1, 2)
    parts = {"q": x[:, :H], "k": x[:, H:H + G], "v": x[:, H + G:]}
    w = {n: (1 + 0.3 * torch.randn(dim, device="cuda", generator=g)) if affine else None for n in ("q", "k")}
    b = {n: (0.2 * torch.randn(dim, device="cuda", generator=g)) if affine else None for n in ("q", "k")}
    pos = torch.randint(0, 5000, (Bn, N, axes), device="cuda", generator=g, dtype=torch.int32)
    plan = R.rope_plan(dim, rot, axes=axes, layout=layout, theta=100.0) if rot else None
    out = {n: torch.full((Bn, h, N, dim), 9.0, device="cuda", dtype=dt) for n, h in (("q", H), ("k", G), ("v", G))}
    R.ress_qk_norm_rope(parts["q"], parts["k"], out["q"], out["k"], parts["v"] if with_v else None,
                        out["v"] if with_v else None,
                        norm={"none": R.NORM_NONE, "rms": R.NORM_RMS, "layer": R.NORM_LAYER}[norm], eps=1e-5,
                        q_weight=w["q"], q_bias=b["q"], k_weight=w["k"], k_bias=b["k"], plan=plan,
                        positions=pos if rot else None, views=views, specials=specials)
    torch.cuda.synchronize()
    assert torch.equal(packed, keep)
    to = torch.tensor(T.tail_order(N, views, specials), device="cuda")
    if with_v:
        assert torch.equal(out["v"][:, :, to], parts["v"])
    else:
        assert bool((out["v"] == 9).all())
    for n in ("q", "k"):
        xd = parts[n].double()
        y, r = T.head_norm(xd, norm, 1e-5, w[n], b[n])
        tol = torch.zeros_like(xd)
        if norm != "none":
            big = float(w[n].abs().max()) if affine else 1.0
            off = float(b[n].abs().max()) if affine else 0.0
            tol = tol + 40 * U * (xd.abs().amax(-1, keepdim=True) * r * big + off)
        if rot:
            f, amp = T.frequencies(rot // axes, 100.0)
            want = T.rope(y, pos, rot, axes, layout, f, amp)
            tol = 2 * tol + 8 * U * _pair_sizes(y, rot, axes, layout)
        else:
            want = y
        tol = tol + _step(want, dt) * (1 + 64 * U)
        err = (out[n][:, :, to].double() - want).abs()
        assert bool((err <= tol).all()), f"{n}: worst {float((err / tol.clamp_min(1e-300)).max()):.2f} of the tolerance"


@pytest.mark.gpu
def test_qk_in_place_zero_rows_and_rows_that_are_not_finite():
    """In place inside the packed projection; a zero row stays finite (eps), and a row with an
    infinity or NaN does not reach the others."""
    packed = torch.randn(2, 40, 6, 64, device="cuda").to(BF16)
    packed[0, 3, 0] = 0
    clean = packed.clone()
    plan = R.rope_plan(64)
    run = lambda p, o: R.ress_qk_norm_rope(  # noqa: E731
        p[:, :, :4].transpose(1, 2), p[:, :, 4:5].transpose(1, 2), o[:, :, :4].transpose(1, 2),
        o[:, :, 4:5].transpose(1, 2), norm=R.NORM_LAYER, plan=plan)
    want = clean.clone()
    run(clean, want)
    assert bool(torch.isfinite(want).all()) and bool((want[0, 3, 0] == 0).all())
    packed[1, 7, 2, 5] = float("inf")
    packed[1, 8, 4, 0] = float("nan")
    run(packed, packed)
    hit = torch.zeros(2, 40, 6, dtype=torch.bool, device="cuda")
    hit[1, 7, 2] = hit[1, 8, 4] = True
    assert torch.equal(packed[~hit], want[~hit])
    assert not bool(torch.isfinite(packed[1, 7, 2]).any())
    assert torch.equal(packed[:, :, 5], clean[:, :, 5])


@pytest.mark.gpu
def test_token_operators_on_a_side_stream_and_in_a_graph():
    packed = torch.randn(1, 300, 12, 64, device="cuda").to(BF16)
    q, k, v = (packed[:, :, 4 * i:4 * i + 4].transpose(1, 2) for i in range(3))
    plan = R.rope_plan(64, axes=2)
    pos = torch.randint(0, 40, (1, 300, 2), device="cuda", dtype=torch.int32)
    outs = [torch.empty(1, 4, 300, 64, device="cuda", dtype=BF16) for _ in range(3)]
    turned = torch.empty_like(outs[0])

    def run(stream=None):
        R.ress_qk_norm_rope(q, k, outs[0], outs[1], v, outs[2], plan=plan, positions=pos, views=3, specials=4,
                            stream=stream)
        R.ress_rope(plan, outs[0], pos, turned, inverse=True, stream=stream)

    run()
    torch.cuda.synchronize()
    want = [x.clone() for x in (*outs, turned)]
    side = torch.cuda.Stream()
    for x in (*outs, turned):
        x.zero_()
    side.wait_stream(torch.cuda.current_stream())
    run(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((*outs, turned), want))
    graph = SparseGlobalAttention.capture(run)
    packed.copy_(packed.flip(1))
    graph.replay()
    torch.cuda.synchronize()
    got = [x.clone() for x in (*outs, turned)]
    assert not torch.equal(got[0], want[0])
    run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((*outs, turned), got))


@pytest.mark.gpu
def test_layer_from_its_packed_projection():
    """prepare() and forward() from [B,N,3,H,64] in view order: the gathers, norm and rotation
    done apart give the same q, k, v, and the layer the same output."""
    wl = W.make_workload(2, heads=4, views=3)
    dev = torch.device("cuda")
    Bn, H, N, _ = wl.q.shape
    views, S = 3, 5
    to = torch.tensor(T.tail_order(N, views, S))
    view_order = [x[:, :, to].to(dev) for x in (wl.q, wl.k, wl.v)]
    packed = torch.stack([x.transpose(1, 2) for x in view_order], 2).contiguous()
    t = torch.arange(N, device=dev)
    grid = torch.stack([t % 37, t // 37 % 37], -1).to(torch.int32)
    plan = R.rope_plan(64, axes=2, theta=100.0)
    layer = SparseGlobalAttention(Bn, H, N, device=dev)
    layer.load_output_projection(wl.w_o.to(dev))
    q, k, v = layer.prepare(packed, plan, grid, norm=R.NORM_RMS, views=views, specials=S)
    normed = [torch.empty_like(x) for x in view_order[:2]]
    R.ress_qk_norm_rope(*view_order[:2], *normed, norm=R.NORM_RMS, plan=plan, positions=grid)
    for got, src in zip((q, k, v), (*normed, view_order[2])):
        want = torch.empty_like(src)
        R.ress_token_gather(layer.shape, views, S, False, src.contiguous(), want)
        assert torch.equal(got, want)
    args = (wl.method, wl.budgets, wl.keep_k.to(dev), wl.dense_q.to(dev), wl.rounds, wl.rho, wl.eps, wl.select_seed)
    out = layer.forward(q, k, v, *args).clone()
    ref = SparseGlobalAttention(Bn, H, N, device=dev)
    ref.load_output_projection(wl.w_o.to(dev))
    assert torch.equal(out, ref.forward(q.clone(), k.clone(), v.clone(), *args))
    assert layer.device_error() == 0
    with pytest.raises(ValueError):
        layer.prepare(packed[:, :-1])
