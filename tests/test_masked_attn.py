"""Attention over kept blocks with changed scores (ress_masked_attn) against 64 bits.

Tolerances.  A score is a sum of 64 exact products in fp32, each addition off by at most one
step: 64 * 2^-23 of sum|q k| scale.  A cap keeps that (its slope is at most 1) and adds the
tanh's own error: below c 2^-20, and below 2^-20 of the largest score where all stay under
the cap (its polynomials are relative); bias and scale round three times.  Call their sum e.  lse is
off by at most e, the exponentials (2^-21), the sum (2^-23 a tile, as the sums of a tile are
trees) and its own rounding.  A weight is off by 2 e and by its rounding to bf16 (2^-8), the
products' sum by 2^-23 a key, and the output rounds once (2^-8):
    |out - exact| <= (2^-8 + 2 e + (N + 64) 2^-23) sum w|v| + 2^-8 |out|.
"""
import ctypes
import math

import pytest
import torch

from block_sparse_global_b200 import build as B
from block_sparse_global_b200 import ress as R
from block_sparse_global_b200.pipeline import SparseGlobalAttention
from oracle import token_oracle as T

INVALID, UNSUPPORTED, OK = 1, 2, 0
FAKE = 0x7F0000000000
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return R.load()


# ------------------------------------------------------------------------ on the host
def test_refusals(lib):
    def call(shape=None, mods=None, q=FAKE, k=FAKE, v=FAKE, idx=FAKE, cnt=FAKE, order=None, scale=0.125, out=FAKE,
             lse=None, ws=FAKE, ws_bytes=1 << 40, err=None, **m):
        s = shape or R.make_shape(1, 2, 1000)
        p = R.ress_attn_mods(m.pop("q_len", 1000))
        for n, x in m.items():
            setattr(p, n, x)
        return lib.ress_masked_attn(ctypes.byref(s), ctypes.byref(p), q, k, v, idx, cnt, order, scale, out, lse, ws,
                                    ws_bytes, err, None)

    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(ws=None), dict(idx=None),
                dict(cnt=None), dict(q=FAKE + 8), dict(out=FAKE + 2), dict(idx=FAKE + 4), dict(order=FAKE + 8),
                dict(lse=FAKE + 2), dict(err=FAKE + 1), dict(ws=FAKE + 8), dict(scale=0.0), dict(scale=-1.0),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(softcap=-1.0),
                dict(softcap=float("nan")), dict(softcap=float("inf")), dict(softcap=1e-30),
                dict(softcap=1e31), dict(softcap=1e25), dict(scale=2e30), dict(q_len=-1), dict(slopes=FAKE),
                dict(slopes=FAKE + 2, q_pos=FAKE, k_pos=FAKE), dict(q_pos=FAKE), dict(k_pos=FAKE), dict(q_doc=FAKE),
                dict(k_doc=FAKE), dict(q_order=FAKE), dict(k_order=FAKE), dict(q_doc=FAKE + 1, k_doc=FAKE),
                dict(q_order=FAKE, k_order=FAKE + 2)):
        assert call(**bad) == INVALID, bad
    s = R.make_shape(1, 2, 1000)
    need = R.ress_masked_attn_workspace_bytes(s, 1000)
    assert need > 0 and call(ws_bytes=need - 1) == INVALID
    assert call(shape=R.make_shape(1, 2, 1000, head_dim=128)) == UNSUPPORTED
    assert call(q_len=4096 * 128 + 1) == UNSUPPORTED
    assert lib.ress_masked_attn(None, None, *([FAKE] * 6), 0.125, FAKE, None, FAKE, 1 << 40, None, None) == INVALID
    nothing = dict(q=None, k=None, v=None, out=None, ws=None, ws_bytes=0)
    assert call(q_len=0, **nothing) == OK
    assert call(shape=R.make_shape(0, 2, 1000), **nothing) == OK
    assert R.ress_masked_attn_workspace_bytes(s, 0) == 0
    assert R.ress_masked_attn_workspace_bytes(R.make_shape(1, 2, 0), 5) == 0
    assert R.ress_masked_attn_workspace_bytes(s, -3) == 0


def test_binding_refuses_what_does_not_fit():
    s = R.make_shape(1, 2, 300)
    k = torch.zeros(1, 2, 300, 64, dtype=BF16)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    i32 = dict(dtype=torch.int32)

    def call(q=k, kk=k, out=k, idx=None, cnt=None, order=None, **kw):
        R.ress_masked_attn(s, q, kk, k, idx, cnt, order, 0.125, out, workspace=ws, **kw)

    for bad in (dict(q=k.float()), dict(q=k[:, :1]), dict(q=k[0]), dict(kk=k[:, :, :299]), dict(out=k[:, :, :299]),
                dict(q=k.transpose(1, 2).contiguous().transpose(1, 2)),
                dict(idx=torch.zeros(1, 2, 3, 2, **i32), cnt=torch.zeros(1, 2, 3, **i32)),
                dict(idx=torch.zeros(1, 2, 3, 3, **i32), cnt=torch.zeros(1, 2, 2, **i32)),
                dict(order=torch.zeros(5, **i32)), dict(slopes=torch.zeros(3)),
                dict(q_doc=torch.zeros(1, 299, **i32), k_doc=torch.zeros(1, 300, **i32)),
                dict(q_doc=torch.zeros(1, 300), k_doc=torch.zeros(1, 300)),
                dict(q_order=torch.zeros(300, **i32), k_order=torch.zeros(300, **i32)),
                dict(lse=torch.zeros(1, 2, 299)),
                dict()):                                      # all fits, but not on a GPU
        with pytest.raises(ValueError):
            call(**bad)


# ------------------------------------------------------------------------- on the GPU
def _run(q, k, v, key_block=128, lists=None, scale=0.125, order=None, lse=True, dev_err=None, stream=None, out=None,
         workspace=None, **mods):
    Bn, H, Nq, _ = q.shape
    N = k.shape[2]
    shape = R.make_shape(Bn, H, N, key_block=key_block)
    nq, nk = (Nq + 127) // 128, R.grid(N, key_block)[1]
    idx = cnt = None
    if lists is not None:
        idx = torch.full((Bn, H, nq, nk), -77, dtype=torch.int32)     # past kv_cnt: never looked at
        cnt = torch.zeros(Bn, H, nq, dtype=torch.int32)
        for (b, h, i), row in lists.items():
            idx[b, h, i, :len(row)] = torch.tensor(row, dtype=torch.int32)
            cnt[b, h, i] = len(row)
        idx, cnt = idx.cuda(), cnt.cuda()
    if workspace is None:
        workspace = torch.empty(max(16, R.ress_masked_attn_workspace_bytes(shape, Nq)), dtype=torch.uint8,
                                device="cuda").fill_(255)             # NaNs where nothing was written
    out = torch.full((Bn, H, Nq, 64), 3.0, dtype=BF16, device="cuda") if out is None else out
    l = torch.full((Bn, H, Nq), 3.0, device="cuda") if lse else None
    R.ress_masked_attn(shape, q, k, v, idx, cnt, order, scale, out, l, workspace=workspace, dev_err=dev_err,
                       stream=stream, **mods)
    return out, l


def _check(q, k, v, out, lse, key_block=128, lists=None, scale=0.125, **mods):
    want, want_lse, size, reach = T.masked_attn(q, k, v, scale, key_block, lists, **mods)
    N = k.shape[2]
    far = 0.0
    if mods.get("slopes") is not None and N and q.shape[2]:
        span = (mods["q_pos"].double().amax() - mods["k_pos"].double().amin()).abs() + \
               (mods["k_pos"].double().amax() - mods["q_pos"].double().amin()).abs()
        far = float(span * mods["slopes"].abs().max())
    cap = min(mods.get("softcap", 0.0), float(reach.max()) if reach.numel() else 0.0)
    e = 64 * 2.0 ** -23 * reach + cap * 2.0 ** -20 + 4 * 2.0 ** -24 * (reach + far)
    none = want_lse == -math.inf
    assert bool((lse[none] == -math.inf).all()) and bool((out[none] == 0).all())
    seen = ~none
    tol = e + 2.0 ** -20 + (N / 128 + 8) * 2.0 ** -23 + 2.0 ** -22 * want_lse.abs()
    err = (lse.double() - want_lse).abs()
    assert bool((err[seen] <= tol[seen]).all()), f"lse: worst {float((err / tol)[seen].max()):.2f} of the tolerance"
    tol = (2.0 ** -8 + 2 * e + (N + 64) * 2.0 ** -23).unsqueeze(-1) * size + 2.0 ** -8 * want.abs() + 1e-30
    err = (out.double() - want).abs()
    assert bool((err <= tol).all()), f"out: worst {float((err / tol).max()):.2f} of the tolerance"


def _inputs(Bn, H, N, Nq, seed=0, size=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    mk = lambda n: (size * torch.randn(Bn, H, n, 64, device="cuda", generator=g)).to(BF16)  # noqa: E731
    return mk(Nq), mk(N), mk(N), g


def _arrays(Bn, N, Nq, docs, pad, order, bias, H, g, shuffle=False):
    """q_* is the end of k_* where Nq <= N, else its own."""
    t = torch.arange(N)
    m = {}
    last = slice(N - Nq, N) if Nq <= N else None

    def pair(name, x):
        x = x.to(torch.int32).expand(Bn, N).clone()
        if shuffle:
            x = torch.stack([row[torch.randperm(N)] for row in x])
        qx = x[:, last] if last is not None else x[:, torch.arange(Nq) % N]
        m["k_" + name], m["q_" + name] = x.cuda(), qx.contiguous().cuda()

    if docs:
        d = t * docs // max(1, N - pad)
        d[N - pad:] = -1
        d[t >= N - pad // 2] = -2
        pair("doc", d)
    if order == "token":
        pair("order", t)
    elif order == "prefix":
        pair("order", (t - N // 3 + 1).clamp_min(0))
    elif order == "view":
        pair("order", t // 100)
    if bias:
        pair("pos", t)
        m["slopes"] = bias * torch.pow(2.0, -8.0 * torch.arange(1, H + 1, device="cuda") / H)
    return m


CASES = [  # B, H, N, Nq, key_block, keep, softcap, docs, pad, order, bias
    (1, 1, 1, 1, 128, 1.0, 0.0, 0, 0, "none", 0.0), (2, 3, 1, 200, 64, 1.0, 30.0, 0, 0, "none", 0.0),
    (1, 2, 127, 127, 128, 1.0, 0.0, 0, 0, "token", 0.0), (1, 2, 65, 65, 64, 1.0, 0.0, 0, 0, "token", 0.1),
    (1, 4, 1024, 1024, 128, 1.0, 0.0, 0, 0, "prefix", 0.0), (2, 2, 700, 700, 128, 0.5, 0.0, 3, 50, "none", 0.0),
    (2, 3, 1000, 1000, 64, 0.4, 20.0, 5, 90, "view", 0.0), (1, 2, 600, 600, 64, 1.0, 0.0, 2, 600, "none", 0.0),
    (1, 16, 3000, 1, 128, 1.0, 30.0, 0, 0, "token", 0.0), (3, 2, 5000, 1, 64, 1.0, 0.0, 2, 10, "token", 0.01),
    (1, 2, 9000, 7, 128, 0.5, 0.0, 0, 0, "view", 0.0), (1, 8, 2050, 131, 64, 0.3, 50.0, 0, 0, "none", 0.5),
    (1, 2, 300, 900, 128, 1.0, 0.0, 2, 20, "token", 0.0), (1, 40, 1500, 1500, 128, 0.6, 0.0, 0, 0, "view", 0.02),
    (2, 20, 1111, 1111, 64, 1.0, 15.0, 4, 101, "token", 0.0), (1, 1, 20000, 33, 128, 1.0, 200.0, 0, 0, "token", 0.0),
    (1, 3, 900, 900, 128, 0.0, 0.0, 0, 0, "none", 0.0), (1, 24, 1800, 1800, 64, 0.5, 0.0, 0, 0, "token", 0.0)]


def _lists(Bn, H, Nq, N, key_block, keep, g):
    if keep >= 1.0:
        return None
    nq, nk = (Nq + 127) // 128, (N + key_block - 1) // key_block
    out = {}
    for b in range(Bn):
        for h in range(H):
            for i in range(nq):
                n = max(0, min(nk, round(keep * nk) + (h + i) % 3 - 1)) if keep else 0
                out[(b, h, i)] = torch.randperm(nk)[:n].tolist()      # any order
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("shuffle", [False, True])
@pytest.mark.parametrize("Bn,H,N,Nq,kb,keep,cap,docs,pad,order,bias", CASES)
def test_against_64_bits(Bn, H, N, Nq, kb, keep, cap, docs, pad, order, bias, shuffle):
    torch.manual_seed(N + Nq)
    q, k, v, g = _inputs(Bn, H, N, Nq, seed=N, size=1.5)
    lists = _lists(Bn, H, Nq, N, kb, keep, g)
    mods = _arrays(Bn, N, Nq, docs, pad, order, bias, H, g, shuffle)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = _run(q, k, v, kb, lists, dev_err=err, softcap=cap, **mods)
    torch.cuda.synchronize()
    assert int(err) == 0
    _check(q, k, v, out, lse, kb, lists, softcap=cap, **mods)
    again, lse2 = _run(q, k, v, kb, lists, softcap=cap, **mods)       # the same bits
    assert torch.equal(again, out) and torch.equal(lse2, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("Bn,H,N,Nq,kb,keep,cap,docs,pad,order,bias", [
    (1, 16, 8000, 8000, 128, 0.5, 0.0, 3, 150, "none", 0.0), (2, 6, 7777, 7777, 64, 0.5, 30.0, 2, 33, "token", 0.01),
    (1, 20, 7000, 7000, 128, 0.3, 0.0, 0, 0, "view", 0.0),
    (1, 16, 9000, 1500, 128, 0.5, 0.0, 2, 100, "token", 0.0), (1, 16, 9001, 1374, 64, 0.25, 0.0, 0, 0, "view", 0.02)])
def test_many_rows_and_long_rows(Bn, H, N, Nq, kb, keep, cap, docs, pad, order, bias):
    """Rows enough to be put in order by what they see, and rows long enough for several parts."""
    torch.manual_seed(N)
    q, k, v, g = _inputs(Bn, H, N, Nq, seed=N)
    lists = _lists(Bn, H, Nq, N, kb, keep, g)
    mods = _arrays(Bn, N, Nq, docs, pad, order, bias, H, g)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = _run(q, k, v, kb, lists, dev_err=err, softcap=cap, **mods)
    assert int(err) == 0
    _check(q, k, v, out, lse, kb, lists, softcap=cap, **mods)


@pytest.mark.gpu
@pytest.mark.parametrize("size", [0.05, 6.0, 40.0])
@pytest.mark.parametrize("cap", [0.0, 1e-3, 5.0, 50.0, 1e5, 1e15])
def test_small_large_and_saturated_scores(size, cap):
    q, k, v, g = _inputs(1, 2, 500, 500, seed=7, size=size)
    out, lse = _run(q, k, v, softcap=cap)
    _check(q, k, v, out, lse, softcap=cap)


@pytest.mark.gpu
@pytest.mark.parametrize("kb", [64, 128])
@pytest.mark.parametrize("cap", [0.0, 25.0])
@pytest.mark.parametrize("kind", ["view", "stride", "backwards", "far", "ahead", "two rates", "random"])
def test_positions_of_every_kind(kind, cap, kb):
    """Positions that run evenly, stand still, jump inside a tile or lie in any order, behind
    and ahead of the queries."""
    N = 700
    t = torch.arange(N)
    pos = {"view": t // 90, "stride": 3 * t, "backwards": 5000 - t, "far": t + (1 << 24) - 900, "ahead": t + 10000,
           "two rates": torch.where(t < 330, t, 4 * t), "random": torch.randint(-2000, 2000, (N,))}[kind]
    pos = pos.to(torch.int32).view(1, N).cuda()
    q, k, v, g = _inputs(1, 3, N, N, seed=13)
    qp = t.to(torch.int32).view(1, N).cuda() if kind == "ahead" else pos
    slopes = torch.tensor([0.02, -0.01, 0.0005], device="cuda")
    lists = _lists(1, 3, N, N, kb, 0.6, g)
    mods = dict(slopes=slopes, q_pos=qp, k_pos=pos)
    out, lse = _run(q, k, v, kb, lists, softcap=cap, **mods)
    _check(q, k, v, out, lse, kb, lists, softcap=cap, **mods)


@pytest.mark.gpu
def test_plain_call_agrees_with_the_unmasked_kernel():
    q, k, v, g = _inputs(1, 6, 1900, 1900, seed=3)
    lists = _lists(1, 6, 1900, 1900, 128, 0.4, g)
    out, lse = _run(q, k, v, 128, lists)
    _check(q, k, v, out, lse, 128, lists)
    layer = SparseGlobalAttention(1, 6, 1900)
    for r, row in lists.items():
        layer.kv_idx[r][:len(row)] = torch.tensor(row, dtype=torch.int32)
        layer.kv_cnt[r] = len(row)
    layer.attend(q, k, v)
    seen = lse > -math.inf
    assert float((layer.out.float() - out.float()).abs().max()) <= 2e-2      # the bars of the unmasked
    assert float((layer.lse - lse)[seen].abs().max()) <= 1e-3                # kernel's own parity tests
    R.ress_attn_schedule(layer.shape, layer.kv_cnt, layer.order)
    sched, lse2 = _run(q, k, v, 128, lists, order=layer.order)
    assert torch.equal(sched, out) and torch.equal(lse2, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("kb", [64, 128])
@pytest.mark.parametrize("Nq", [400, 3, 1])
def test_hidden_keys_hold_anything(kb, Nq):
    """Infinities and NaN in keys and values that the masks hide do not change a bit of the
    other rows; where a row sees them, its output says so; padded queries may hold them too."""
    q, k, v, g = _inputs(1, 3, 400, Nq, seed=11)
    mods = _arrays(1, 400, Nq, 2, 40, "token", 0.0, 3, g)
    clean, lse = _run(q, k, v, kb, **mods)
    _check(q, k, v, clean, lse, kb, **mods)
    k2, v2 = k.clone(), v.clone()
    for bad, at in ((float("nan"), 362), (float("inf"), 370), (-float("inf"), 399)):   # padding: seen by none
        k2[:, :, at] = bad
        v2[:, :, at, ::3] = bad
    q2 = q.clone()
    if Nq == 400:
        q2[:, :, 365] = float("nan")
    out, lse2 = _run(q2, k2, v2, kb, **mods)
    assert torch.equal(out, clean) and torch.equal(lse2, lse)
    v2[:, :, 300, 5] = float("inf")          # document 1, seen by its later tokens only
    v2[:, :, 301, 6] = float("nan")
    out, _ = _run(q2, k2, v2, kb, **mods)
    if Nq == 400:
        rows = torch.arange(400, device="cuda")
        sees = (rows >= 300) & (rows < 360)
        assert torch.equal(out[:, :, ~sees], clean[:, :, ~sees])
        assert bool((out[:, :, 300:360, 5] == float("inf")).all())
        assert bool(torch.isnan(out[:, :, 301:360, 6]).all()) and bool(torch.isfinite(out[:, :, 300, 6]).all())
        same = torch.ones(64, dtype=torch.bool, device="cuda")
        same[5] = same[6] = False
        assert torch.equal(out[..., same], clean[..., same])


@pytest.mark.gpu
@pytest.mark.parametrize("kb", [64, 128])
def test_hidden_keys_in_joined_parts(kb):
    """The same where parts of a row are joined: only the part that holds them walks again."""
    N, Nq = 9000, 200
    q, k, v, g = _inputs(1, 3, N, Nq, seed=17)
    mods = _arrays(1, N, Nq, 0, 0, "view", 0.0, 3, g)
    clean, lse = _run(q, k, v, kb, **mods)
    _check(q, k, v, clean, lse, kb, **mods)
    v2, k2 = v.clone(), k.clone()
    v2[:, :, 8950:] = float("nan")           # the last view: hidden from the queries before it
    k2[:, :, 8950:] = float("inf")
    v2[:, :, 77, 9] = float("inf")           # seen by all, in the first part
    out, lse2 = _run(q, k2, v2, kb, **mods)
    before = mods["q_order"][0] < 89
    assert bool((out[:, :, before, 9] == float("inf")).all())
    same = torch.ones(64, dtype=torch.bool, device="cuda")
    same[9] = False
    assert torch.equal(out[:, :, before][..., same], clean[:, :, before][..., same])
    assert torch.equal(lse2[:, :, before], lse[:, :, before])


@pytest.mark.gpu
def test_first_tile_of_a_row_holds_an_infinity():
    """The values of the first tile are added by hand before any product ran."""
    q, k, v, g = _inputs(2, 2, 260, 260, seed=5)
    mods = _arrays(2, 260, 260, 0, 0, "token", 0.0, 2, g)
    clean, _ = _run(q, k, v, **mods)
    v2 = v.clone()
    v2[:, :, 4, 63] = -float("inf")
    v2[:, :, 200, 0] = float("inf")
    out, _ = _run(q, k, v2, **mods)
    assert bool((out[:, :, 4:, 63] == -float("inf")).all()) and bool((out[:, :, 200:, 0] == float("inf")).all())
    assert torch.equal(out[..., 1:63], clean[..., 1:63])
    assert torch.equal(out[:, :, :4], clean[:, :, :4]) and torch.equal(out[:, :, :200, 0], clean[:, :, :200, 0])


@pytest.mark.gpu
@pytest.mark.parametrize("N,Nq", [(0, 5), (0, 300), (129, 129)])
def test_rows_without_keys(N, Nq):
    q, k, v, g = _inputs(2, 2, N, Nq)
    mods = {}
    if N:
        far = torch.full((2, N), 9, dtype=torch.int32, device="cuda")
        mods = dict(q_doc=far, k_doc=far + 1)
    out, lse = _run(q, k, v, **mods)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


@pytest.mark.gpu
@pytest.mark.parametrize("kb", [64, 128])
@pytest.mark.parametrize("Bn,H,N", [(1, 1, 1), (1, 1, 70), (2, 3, 129), (1, 16, 2500), (5, 16, 1111), (20, 16, 300),
                                    (1, 8, 20001), (1, 2, 30000)])
@pytest.mark.parametrize("what", ["plain", "masks", "bias"])
def test_single_tokens(Bn, H, N, kb, what):
    """One query per head: lists in any order, masks in any order, values hidden or not."""
    torch.manual_seed(N + H)
    q, k, v, g = _inputs(Bn, H, N, 1, seed=N + Bn, size=1.5)
    lists = _lists(Bn, H, 1, N, kb, 0.6, g) if what != "bias" else None
    mods, cap = {}, 0.0
    if what == "masks":
        mods = _arrays(Bn, N, 1, 2, N // 9, "view", 0.0, H, g, shuffle=True)
        mods["q_doc"] = torch.zeros(Bn, 1, dtype=torch.int32, device="cuda")
        hide = mods["k_doc"] != 0
        k = torch.where(hide[:, None, :, None], torch.full_like(k, float("nan")), k)
        v = torch.where(hide[:, None, :, None], torch.full_like(v, float("inf")), v)
        cap = 8.0
    elif what == "bias":
        mods = _arrays(Bn, N, 1, 0, 0, "none", 0.02, H, g)
    out, lse = _run(q, k, v, kb, lists, softcap=cap, **mods)
    _check(q, k, v, out, lse, kb, lists, softcap=cap, **mods)


@pytest.mark.gpu
def test_a_block_listed_twice_counts_twice():
    q, k, v, g = _inputs(1, 2, 640, 640, seed=2)
    lists = {(0, h, i): [1, 3, 1] if h else [4, 4, 4, 0, 4] for h in range(2) for i in range(5)}
    out, lse = _run(q, k, v, 128, lists)
    _check(q, k, v, out, lse, 128, lists)


@pytest.mark.gpu
@pytest.mark.parametrize("Nq", [600, 300, 2, 1])
def test_bad_lists_set_the_error_and_leave_the_row(Nq):
    """An index or a count out of range is found by the kernel's own check before any load."""
    N = {600: 600, 300: 9000}.get(Nq, 1100)       # the second in parts that are joined
    q, k, v, g = _inputs(1, 30, N, Nq)
    nq, nk = (Nq + 127) // 128, (N + 127) // 128
    shape = R.make_shape(1, 30, N)
    idx = torch.arange(nk, dtype=torch.int32).expand(1, 30, nq, nk).contiguous().cuda()
    cnt = torch.full((1, 30, nq), nk, dtype=torch.int32, device="cuda")
    idx[0, 3, 0, 2] = nk
    idx[0, 4, 0, 4] = -1
    cnt[0, 5, 0] = nk + 1
    cnt[0, 6, 0] = -2
    ws = torch.empty(R.ress_masked_attn_workspace_bytes(shape, Nq), dtype=torch.uint8, device="cuda")
    out = torch.full((1, 30, Nq, 64), 3.0, dtype=BF16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    R.ress_masked_attn(shape, q, k, v, idx, cnt, None, 0.125, out, workspace=ws, dev_err=err)
    torch.cuda.synchronize()
    assert int(err) == 4
    rows = min(Nq, 128)
    assert bool((out[0, 3:7, :rows] == 3).all())
    want, _ = _run(q, k, v)
    good = [h for h in range(30) if h not in (3, 4, 5, 6)]
    assert torch.equal(out[0, good], want[0, good]) and torch.equal(out[0, :, rows:], want[0, :, rows:])


@pytest.mark.gpu
def test_new_tokens_over_a_cache():
    """All tokens, single ones and a chunk over the same keys; the queries' arrays are the ends
    of the keys' (off the 16-byte boundary)."""
    q, k, v, g = _inputs(1, 4, 520, 520, seed=9)
    t = torch.arange(520, dtype=torch.int32, device="cuda").view(1, 520)
    for lo, hi in ((0, 520), (0, 1), (300, 301), (519, 520), (256, 520)):
        mods = dict(q_order=t[:, lo:hi], k_order=t, softcap=30.0, slopes=torch.full((4,), 0.05, device="cuda"),
                    q_pos=t[:, lo:hi], k_pos=t)
        out, l = _run(q[:, :, lo:hi].contiguous(), k, v, **mods)
        _check(q[:, :, lo:hi], k, v, out, l, **mods)


@pytest.mark.gpu
def test_guards_streams_and_graphs_with_their_own_workspaces():
    """Two calls at once on two streams, captured and replayed on new data; memory around the
    outputs stays."""
    sets = []
    for i, (N, Nq) in enumerate(((3000, 2), (777, 777), (9000, 200))):
        q, k, v, g = _inputs(1, 3, N, Nq, seed=20 + i)
        mods = _arrays(1, N, Nq, 2, 9, "token", 0.0, 3, g)
        room = torch.full((3 * Nq * 64 + 128,), 5.0, dtype=BF16, device="cuda")
        out = room[64:-64].view(1, 3, Nq, 64)
        ws = torch.empty(R.ress_masked_attn_workspace_bytes(R.make_shape(1, 3, N), Nq), dtype=torch.uint8, device="cuda")
        sets.append((q, k, v, mods, room, out, ws))
    want = [_run(q, k, v, lse=False, **m)[0] for q, k, v, m, *_ in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (q, k, v, m, room, out, ws) in zip(streams, sets):
            _run(q, k, v, lse=False, out=out, workspace=ws, stream=s, **m)
    torch.cuda.synchronize()
    for w, (q, k, v, m, room, out, ws) in zip(want, sets):
        assert torch.equal(out, w)
        assert bool((room[:64] == 5).all()) and bool((room[-64:] == 5).all())

    def both():
        for q, k, v, m, room, out, ws in sets:
            shape = R.make_shape(1, 3, k.shape[2])
            R.ress_masked_attn(shape, q, k, v, None, None, None, 0.125, out, workspace=ws, **m)

    graph = SparseGlobalAttention.capture(both)
    for q, k, v, *_ in sets:
        q.copy_(-q)
        v.copy_(v.flip(2))
    graph.replay()
    torch.cuda.synchronize()
    for q, k, v, m, room, out, ws in sets:
        assert torch.equal(out, _run(q, k, v, lse=False, **m)[0])


@pytest.mark.gpu
@pytest.mark.parametrize("key_block", [128, 64])
def test_layer_with_masks_from_projection_to_new_tokens(key_block):
    """A run of the operators as a layer uses them: packed projection -> norm, rotation and
    tail order -> selection -> capped attention, causal over views, then one new token over
    the layer's keys as a cache."""
    views, per, S, H = 3, 260, 4, 4
    N = views * per
    g = torch.Generator(device="cuda").manual_seed(4)
    packed = torch.randn(1, N, 3, H, 64, device="cuda", generator=g).to(BF16)
    layer = SparseGlobalAttention(1, H, N, key_block=key_block)
    layer.load_output_projection(torch.randn(64 * H, 64 * H, device="cuda", generator=g) / 16)
    plan = R.rope_plan(64)
    q, k, v = layer.prepare(packed, plan, norm=R.NORM_RMS, views=views, specials=S)
    view = torch.empty(N, dtype=torch.int32)
    view[torch.tensor(T.tail_order(N, views, S))] = (torch.arange(N) // per).to(torch.int32)
    view = view.view(1, N).cuda()
    mods = dict(softcap=20.0, q_order=view, k_order=view)
    nk = layer.nk
    out = layer.forward(q, k, v, R.SELECT_DRIFT, [nk // 2] * H, rounds=2, mods=mods)
    torch.cuda.synchronize()
    assert layer.device_error() == 0
    _check(q, k, v, out, layer.lse, key_block, layer.kept_lists(), **mods)
    new = torch.randn(1, H, 1, 64, device="cuda", generator=g).to(BF16)
    turned = torch.empty_like(new)
    R.ress_rope(plan, new, torch.tensor([N], dtype=torch.int32, device="cuda"), turned)
    step = dict(softcap=20.0, q_order=torch.tensor([[1]], dtype=torch.int32, device="cuda"), k_order=view)
    lse = torch.empty(1, H, 1, device="cuda")
    got = layer.attend_masked(turned, k, v, kept=False, lse=lse, **step)
    assert got.shape == (1, H, 1, 64)
    _check(turned, k, v, got, lse, key_block, **step)
    with pytest.raises(ValueError):
        layer.attend_masked(turned, k, v)


@pytest.mark.gpu
def test_order_that_is_no_permutation_sets_the_error():
    """An entry of work_order out of range is found by the kernel's own check."""
    q, k, v, g = _inputs(1, 40, 500, 500)       # 160 rows: one CTA each
    order = torch.arange(160, dtype=torch.int32, device="cuda")
    want, _ = _run(q, k, v)
    order[3], order[5] = 160, -1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, _ = _run(q, k, v, order=order, dev_err=err)
    torch.cuda.synchronize()
    assert int(err) == 4
    assert bool((out[0, 0, 384:] == 3).all()) and bool((out[0, 1, 128:256] == 3).all())
    assert torch.equal(out[0, 2:], want[0, 2:]) and torch.equal(out[0, 0, :384], want[0, 0, :384])


@pytest.mark.gpu
def test_layer_graph_of_new_tokens_outlives_larger_calls():
    """A captured call keeps its workspace when later calls of the layer need larger ones."""
    layer = SparseGlobalAttention(1, 4, 9000)
    q, k, v, g = _inputs(1, 4, 9000, 200, seed=30)
    out = torch.empty(1, 4, 200, 64, dtype=BF16, device="cuda")
    graph = layer.capture(lambda: layer.attend_masked(q, k, v, kept=False, out=out, softcap=20.0))
    big = torch.randn(1, 4, 2000, 64, device="cuda").to(BF16)
    layer.attend_masked(big, k, v, kept=False)
    junk = [torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
    q.copy_(-q)
    graph.replay()
    torch.cuda.synchronize()
    want, _ = _run(q, k, v, softcap=20.0)
    assert torch.equal(out, want) and len(junk) == 8
