"""What the layer's token operators and masked attention cost, and what they compute.

Three operators around a global-attention layer:

  rope   rotary positions of one [B, H, N, D] tensor (any strides; part of the head; one to
         three position axes; both pair layouts; scaled frequencies), and its inverse
  qk     per-head norm of queries and keys and their rotation in one pass, out of the packed
         projection into the layer's head-major layout (values, and the move of every
         view's special tokens to the tail, in the same pass)
  attn   attention over kept key blocks whose scores are capped by a tanh, lowered with the
         distance and masked by document and by order, for all tokens or for the newest

`own` chooses between the plain torch form and this package's entry points.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
VIEW = 1374          # tokens of a view: 5 special and 37 x 37 patch tokens
VIEW_SPECIAL = 5
GRID = 37


# ------------------------------------------------------------------------------- cases
def _case(c, kw):
    c.update(kw)
    if c["name"] is None:  # a drawn case has none
        del c["name"]
    return c


def _rope(name, **kw):
    c = dict(name=name, op="rope", batch=1, heads=16, tokens=1, dim=64, rot=64, axes=1, layout="half",
             dtype="bf16", order="bhnd", theta=10000.0, scaling="none", factor=1.0, original=0,
             inverse=False, far=100000)
    return _case(c, kw)


def _qk(name, **kw):
    c = dict(name=name, op="qk", batch=1, heads=16, kv_heads=16, tokens=1, dim=64, rot=64, axes=1,
             layout="half", dtype="bf16", theta=10000.0, scaling="none", factor=1.0, original=0,
             norm="rms", affine=True, with_v=True, views=1, specials=0, far=100000)
    return _case(c, kw)


def _attn(name, **kw):
    c = dict(name=name, op="attn", batch=1, heads=16, tokens=1024, queries=0, key_block=128, keep=1.0,
             softcap=0.0, bias="none", docs=0, pad=0, order="none", prefix=0)
    return _case(c, kw)


def listed():
    return [
        # one new token for each of 16 streams, far along: latency alone
        _rope("rope step", batch=16),
        # keys of a 128-wide head kept in 32 bits, three quarters of it rotated, stretched to
        # eight times the trained length, token-major as the projection wrote them; odd length
        _rope("rope fp32 partial yarn", batch=2, heads=8, tokens=4099, dim=128, rot=96, dtype="fp32",
              order="bnhd", scaling="yarn", factor=8.0, original=4096),
        # the keys of a 100-view layer turned back (the rotation's inverse), adjacent pairs
        _rope("rope 100 views back", tokens=100 * VIEW, dtype="fp16", layout="interleaved",
              scaling="linear", factor=4.0, inverse=True),
        # queries and keys of one new token per stream, four query heads to a key head
        _qk("qk step", batch=8, kv_heads=4),
        # 8-view layer: layer norm, two-axis grid positions, special tokens to the tail
        _qk("qk 8 views", tokens=8 * VIEW, axes=2, theta=100.0, norm="layer", views=8, specials=VIEW_SPECIAL),
        # odd lengths, wide heads, part of the head, adjacent pairs, no values
        _qk("qk odd fp16", batch=3, heads=12, kv_heads=6, tokens=1217, dim=128, rot=48, layout="interleaved",
            dtype="fp16", with_v=False),
        # the 100-view layer's whole projection
        _qk("qk 100 views", tokens=100 * VIEW, axes=2, theta=100.0, norm="layer", views=100,
            specials=VIEW_SPECIAL),
        # one new token over an 8-view cache, capped scores
        _attn("attn step", tokens=8 * VIEW, queries=1, softcap=30.0),
        # the small layer: a prefix that sees itself whole, then token after token
        _attn("attn prefix", heads=4, tokens=1024, order="prefix", prefix=256),
        # several scenes packed into one 8-view sequence with a padded end, half of the blocks kept
        _attn("attn scenes", tokens=8 * VIEW, keep=0.5, docs=3, pad=200),
        # one new view over 32 views, 64-token key blocks, a quarter kept, nearer views first
        _attn("attn new view", tokens=32 * VIEW, queries=VIEW, key_block=64, keep=0.25, bias="view"),
        # 32 views, each seeing itself and the views before it, capped scores
        _attn("attn causal views", tokens=32 * VIEW, order="view", softcap=50.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "qk", "attn", "attn"])
    if op == "attn":
        heads = rng.choice([1, 2, 3, 4, 8, 12, 16])
        batch = rng.choice([1, 1, 2, 3])
        # no more pairs than the largest layer's, and no more scores of one head
        tokens = _log_int(rng, 1, int(32 * VIEW * min(1.0, batch ** -0.5, (8 / (batch * heads)) ** 0.5)))
        queries = rng.choice([0, 0, 1, _log_int(rng, 1, tokens)])
        docs = rng.choice([0, 0, 1, 2, 5])
        order = rng.choice(["none", "token", "prefix", "view"])
        return _attn(None, batch=batch, heads=heads, tokens=tokens, queries=queries,
                     key_block=rng.choice([64, 128]), keep=rng.choice([1.0, 0.75, 0.5, 0.25, 0.1]),
                     softcap=rng.choice([0.0, 0.0, 15.0, 30.0, 50.0, 200.0]),
                     bias=rng.choice(["none", "none", "token", "view"]), docs=docs,
                     pad=rng.randint(0, tokens // 4) if docs else 0, order=order,
                     prefix=rng.randint(0, tokens) if order == "prefix" else 0)
    dim = rng.choice([32, 64, 64, 80, 96, 128, 256])
    axes = rng.choice([1, 1, 2, 3])
    rot = 2 * axes * rng.randint(2, dim // (2 * axes))
    if rng.random() < 0.5:
        rot = 16 * axes * max(1, rot // (16 * axes)) if 16 * axes <= dim else rot
    scaling = rng.choice(["none", "none", "linear", "ntk", "yarn"])
    common = dict(dim=dim, rot=rot, axes=axes, layout=rng.choice(["half", "interleaved"]),
                  dtype=rng.choice(["bf16", "fp16", "fp32"]), theta=rng.choice([100.0, 10000.0, 500000.0]),
                  scaling=scaling, factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 40.0]),
                  original=rng.choice([2048, 4096, 8192]) if scaling == "yarn" else 0,
                  far=_log_int(rng, 1000, 4000000), batch=_log_int(rng, 1, 16))
    heads = rng.choice([1, 2, 5, 8, 12, 16])
    room = 100 * VIEW * 16 * 64 // (common["batch"] * heads * dim * (2 if common["dtype"] == "fp32" else 1))
    tokens = _log_int(rng, 1, max(1, room))
    if op == "rope":
        return _rope(None, heads=heads, tokens=tokens, order=rng.choice(["bhnd", "bnhd"]),
                     inverse=rng.random() < 0.3, **common)
    kv_heads = rng.choice([h for h in (1, 2, 5, 8, 12, 16) if heads % h == 0])
    views = rng.choice([1, 1, 2, 7])
    tokens = views * max(1, tokens // views)
    return _qk(None, heads=heads, kv_heads=kv_heads, tokens=tokens, norm=rng.choice(["rms", "layer"]),
               affine=rng.random() < 0.8, with_v=rng.random() < 0.6, views=views,
               specials=rng.randint(0, min(5, tokens // views)), **common)


# ------------------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _positions(c, g):
    """int32 [B, N, axes]: streams at places of their own along one axis; a grid of patches, with
    special tokens at 0, along several."""
    B, N, axes = c["batch"], c["tokens"], c["axes"]
    t = torch.arange(N, device="cuda")
    if axes == 1:
        start = torch.randint(0, c["far"], (B, 1), device="cuda", generator=g)
        return (start + t).to(torch.int32).unsqueeze(-1).contiguous()
    s = torch.remainder(t, VIEW) - VIEW_SPECIAL
    p = torch.stack([1 + torch.div(s, GRID, rounding_mode="floor"), 1 + torch.remainder(s, GRID),
                     torch.div(t, VIEW, rounding_mode="floor")][:axes], dim=-1)
    p = torch.where((s < 0).unsqueeze(-1), torch.zeros_like(p), p)
    return p.to(torch.int32).expand(B, N, axes).contiguous()


def _views_base(c, g, n):
    return torch.randn(c["batch"], c["heads"], (n + VIEW - 1) // VIEW, 64, device="cuda", generator=g)


def _tokens_of(c):
    """Per-token int32 rows that the masks and the distance go by, on the host: document (padding
    -1), order, position."""
    N = c["tokens"]
    t = np.arange(N)
    doc = order = pos = None
    if c["docs"]:
        real = N - c["pad"]
        # ragged: the k-th document is about k + 1 times as long as the first
        cuts = np.cumsum(np.arange(1, c["docs"] + 1)) / (c["docs"] * (c["docs"] + 1) / 2) * real
        doc = np.searchsorted(np.floor(cuts), t, side="right")
        doc[real:] = -1
    if c["order"] == "token":
        order = t
    elif c["order"] == "prefix":
        order = np.maximum(0, t - c["prefix"] + 1)
    elif c["order"] == "view":
        order = t // VIEW
    if c["bias"] == "token":
        pos = t
    elif c["bias"] == "view":
        pos = t // VIEW
    return doc, order, pos


def _budgets(c, nk):
    """Kept blocks of each head's rows: around the kept share, from half of it to one and a half."""
    H = c["heads"]
    if c["keep"] >= 1.0:
        return [nk] * H
    return [max(1, min(nk, int(round(c["keep"] * nk * (0.5 + (h + 0.5) / H))))) for h in range(H)]


def prepare(case, seed):
    c, g = case, _gen(seed)
    st = {"case": c}
    if c["op"] == "attn":
        B, H, N, kb = c["batch"], c["heads"], c["tokens"], c["key_block"]
        Nq = c["queries"] or N
        dev = dict(device="cuda", generator=g)
        base = _views_base(c, g, N)
        view = torch.arange(N, device="cuda") // VIEW
        st["k"] = (base[:, :, view] + 0.5 * torch.randn(B, H, N, 64, **dev)).to(torch.bfloat16)
        st["q"] = (base[:, :, view[N - Nq:]] + 0.5 * torch.randn(B, H, Nq, 64, **dev)).to(torch.bfloat16)
        st["v"] = torch.randn(B, H, N, 64, **dev).to(torch.bfloat16)
        for key, x in zip(("doc", "order", "pos"), _tokens_of(c)):
            if x is None:
                st["k_" + key] = st["q_" + key] = None
            else:
                row = torch.from_numpy(x.astype(np.int32)).cuda().expand(B, N).contiguous()
                st["k_" + key], st["q_" + key] = row, row[:, N - Nq:].contiguous()
        st["slopes"] = None
        if c["bias"] != "none":  # a geometric row of slopes, weaker where positions count tokens
            top = 1.0 if c["bias"] == "view" else 0.01
            st["slopes"] = top * torch.pow(2.0, -8.0 * torch.arange(1, H + 1, device="cuda") / H)
        nq, nk = (Nq + 127) // 128, (N + kb - 1) // kb
        st["kv_idx"] = st["kv_cnt"] = None
        if c["keep"] < 1.0:
            cnt = torch.tensor(_budgets(c, nk), device="cuda").view(1, H, 1).expand(B, H, nq)
            rank = torch.rand(B, H, nq, nk, **dev).argsort(-1)
            rank = torch.where(torch.arange(nk, device="cuda") < cnt.unsqueeze(-1), rank, nk)
            st["kv_idx"] = rank.sort(-1).values.clamp_(max=nk - 1).to(torch.int32).contiguous()
            st["kv_cnt"] = cnt.to(torch.int32).contiguous()
        st["scale"] = 0.125
        st["out"] = torch.empty(B, H, Nq, 64, device="cuda", dtype=torch.bfloat16)
        st["lse"] = torch.empty(B, H, Nq, device="cuda")
        if own:  # the shape and the scratch that a layer keeps
            from block_sparse_global_b200 import ress as R
            st["shape"] = R.make_shape(B, H, N, key_block=kb)
            st["workspace"] = torch.empty(R.ress_masked_attn_workspace_bytes(st["shape"], Nq), device="cuda",
                                          dtype=torch.uint8)
        return st
    B, N, D, dt = c["batch"], c["tokens"], c["dim"], DTYPES[c["dtype"]]
    st["positions"] = _positions(c, g)
    if own:  # the frequencies that a model computes once
        from block_sparse_global_b200 import ress as R
        st["plan"] = R.rope_plan(D, c["rot"], axes=c["axes"], layout=c["layout"], theta=c["theta"],
                                 scaling=c["scaling"], factor=c["factor"], original_len=c["original"])
    if c["op"] == "rope":
        H = c["heads"]
        if c["order"] == "bhnd":
            st["x"] = torch.randn(B, H, N, D, device="cuda", generator=g).to(dt)
        else:
            st["x"] = torch.randn(B, N, H, D, device="cuda", generator=g).to(dt).transpose(1, 2)
        st["out"] = torch.empty_like(st["x"])
        return st
    H, G = c["heads"], c["kv_heads"]
    st["packed"] = (torch.randn(B, N, H + 2 * G, D, device="cuda", generator=g)
                    * (0.5 + torch.rand(1, 1, H + 2 * G, 1, device="cuda", generator=g))).to(dt)
    for w in ("q_weight", "k_weight"):
        st[w] = 1 + 0.2 * torch.randn(D, device="cuda", generator=g) if c["affine"] else None
    for w in ("q_bias", "k_bias"):
        st[w] = 0.1 * torch.randn(D, device="cuda", generator=g) if c["affine"] and c["norm"] == "layer" else None
    for n, h in (("q", H), ("k", G), ("v", G)):
        st[n + "_out"] = torch.empty(B, h, N, D, device="cuda", dtype=dt)
    return st


# -------------------------------------------------------------------------- plain forms
def _inverse_frequencies(c):
    """[rot / 2 / axes] in 64 bits, and the factor of cosine and sine."""
    d = c["rot"] // c["axes"]
    i = torch.arange(d // 2, dtype=torch.float64)
    theta, f = c["theta"], c["factor"]
    if c["scaling"] == "ntk":
        theta = theta * f ** (d / (d - 2))
    inv = theta ** (-2 * i / d)
    if c["scaling"] == "linear":
        inv = inv / f
    if c["scaling"] != "yarn":
        return inv, 1.0
    # pairs that turn often within the trained length stay, slow ones are stretched, with a
    # ramp between 32 turns and 1 turn
    at = lambda turns: d * math.log(c["original"] / (turns * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
    low, high = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), d - 1)
    ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
    return inv / f * ramp + inv * (1 - ramp), 0.1 * math.log(f) + 1 if f > 1 else 1.0


def _rotate(c, x, positions, inverse=False):
    """x [B, H, N, D] in 32 bits."""
    B, H, N, D = x.shape
    rot, axes = c["rot"], c["axes"]
    inv, amp = _inverse_frequencies(c)
    angle = positions.double().unsqueeze(-1) * inv.cuda()                    # [B, N, axes, d/2]
    cos, sin = (amp * angle.cos()).float().unsqueeze(1), (amp * angle.sin()).float().unsqueeze(1)
    if inverse:
        sin = -sin
    part = x[..., :rot].reshape(B, H, N, axes, rot // axes)
    if c["layout"] == "half":
        a, b = part.chunk(2, -1)
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned.reshape(B, H, N, rot), x[..., rot:]], -1)


def _norm(c, x, weight, bias):
    if c["norm"] == "layer":
        x = x - x.mean(-1, keepdim=True)
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-5)
    if weight is not None:
        x = x * weight
    return x if bias is None else x + bias


def _to_tail(c, x):
    """Every view's patch tokens first, then every view's special tokens."""
    if c["views"] == 1 and c["specials"] == 0:
        return x
    B, H, N, D = x.shape
    x = x.reshape(B, H, c["views"], N // c["views"], D)
    s = c["specials"]
    return torch.cat([x[:, :, :, s:].reshape(B, H, -1, D), x[:, :, :, :s].reshape(B, H, -1, D)], 2)


def _split(st):
    c = st["case"]
    H, G = c["heads"], c["kv_heads"]
    x = st["packed"].transpose(1, 2)
    return x[:, :H], x[:, H:H + G], x[:, H + G:]


def _plain_qk(st):
    c = st["case"]
    dt = DTYPES[c["dtype"]]
    q, k, v = _split(st)
    out = {}
    for n, x in (("q", q), ("k", k)):
        y = _rotate(c, _norm(c, x.float(), st[n + "_weight"], st[n + "_bias"]), st["positions"])
        out[n] = _to_tail(c, y).to(dt)
    if c["with_v"]:
        out["v"] = _to_tail(c, v).contiguous()
    return out


def _kept(st):
    """[B, H, Nq, N] truth values of the kept block lists, or None."""
    c = st["case"]
    if st["kv_idx"] is None:
        return None
    B, H, nq, nk = st["kv_idx"].shape
    listed_ = torch.arange(nk, device="cuda") < st["kv_cnt"].unsqueeze(-1)
    kept = torch.zeros(B, H, nq, nk, dtype=torch.int32, device="cuda")
    kept = kept.scatter_add_(-1, st["kv_idx"].long(), listed_.int()) > 0
    rows = torch.arange(st["q"].shape[2], device="cuda") // 128
    cols = torch.arange(c["tokens"], device="cuda") // c["key_block"]
    return kept[:, :, rows][..., cols]


def _seen(st):
    """[B, Nq, N] truth values of the document and order masks, or None."""
    seen = None
    if st["k_doc"] is not None:
        qd, kd = st["q_doc"].unsqueeze(2), st["k_doc"].unsqueeze(1)
        seen = (qd == kd) & (qd >= 0)
    if st["k_order"] is not None:
        before = st["k_order"].unsqueeze(1) <= st["q_order"].unsqueeze(2)
        seen = before if seen is None else seen & before
    return seen


def _plain_attn(st):
    c = st["case"]
    seen = _seen(st)
    outs, lses = [], []
    # a head at a time: all heads' scores of the largest layer do not fit the card
    for h in range(c["heads"]):
        one = dict(st, q=st["q"][:, h:h + 1], kv_idx=None)
        if st["kv_idx"] is not None:
            one.update(kv_idx=st["kv_idx"][:, h:h + 1], kv_cnt=st["kv_cnt"][:, h:h + 1])
        s = torch.matmul(st["q"][:, h].float(), st["k"][:, h].float().transpose(1, 2)) * st["scale"]
        if c["softcap"]:
            s = c["softcap"] * torch.tanh(s / c["softcap"])
        if st["slopes"] is not None:
            far = (st["q_pos"].unsqueeze(2) - st["k_pos"].unsqueeze(1)).abs().float()
            s = s - st["slopes"][h] * far
        for mask in (seen, _kept(one)):
            if mask is not None:
                s = s.masked_fill(~mask.reshape(s.shape), -math.inf)
        top = s.amax(-1, keepdim=True)
        top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
        p = torch.exp(s - top)
        total = p.sum(-1, keepdim=True)
        o = torch.matmul(p, st["v"][:, h].float())
        outs.append(torch.where(total > 0, o / total, torch.zeros_like(o)).to(torch.bfloat16))
        lses.append((top + torch.log(total)).squeeze(-1))
    return {"out": torch.stack(outs, 1), "lse": torch.stack(lses, 1)}


# --------------------------------------------------------------------------------- run
def run(state):
    c = state["case"]
    if not own:
        if c["op"] == "attn":
            return _plain_attn(state)
        if c["op"] == "qk":
            return _plain_qk(state)
        return _rotate(c, state["x"].float(), state["positions"], c["inverse"]).to(DTYPES[c["dtype"]])
    from block_sparse_global_b200 import ress as R
    if c["op"] == "rope":
        R.ress_rope(state["plan"], state["x"], state["positions"], state["out"], inverse=c["inverse"])
        return state["out"]
    if c["op"] == "qk":
        q, k, v = _split(state)
        R.ress_qk_norm_rope(q, k, state["q_out"], state["k_out"], v if c["with_v"] else None,
                            state["v_out"] if c["with_v"] else None,
                            norm=R.NORM_LAYER if c["norm"] == "layer" else R.NORM_RMS, eps=1e-5,
                            q_weight=state["q_weight"], q_bias=state["q_bias"], k_weight=state["k_weight"],
                            k_bias=state["k_bias"], plan=state["plan"], positions=state["positions"],
                            views=c["views"], specials=c["specials"])
        return {n: state[n + "_out"] for n in ("q", "k") + (("v",) if c["with_v"] else ())}
    R.ress_masked_attn(state["shape"], state["q"], state["k"], state["v"], state["kv_idx"], state["kv_cnt"],
                       None, state["scale"], state["out"], state["lse"], softcap=c["softcap"],
                       slopes=state["slopes"], q_pos=state["q_pos"], k_pos=state["k_pos"],
                       q_doc=state["q_doc"], k_doc=state["k_doc"], q_order=state["q_order"],
                       k_order=state["k_order"], workspace=state["workspace"])
    return {"out": state["out"], "lse": state["lse"]}


# -------------------------------------------------------------------------------- work
def _pairs(c):
    """Query-key pairs of one head that the masks leave."""
    N, Nq = c["tokens"], c["queries"] or c["tokens"]
    doc, order, _ = _tokens_of(c)
    doc = np.zeros(N, np.int64) if doc is None else doc
    order = np.zeros(N, np.int64) if order is None else order
    total = 0
    for d in np.unique(doc[doc >= 0]):
        mine = np.sort(order[doc == d])
        rows = order[N - Nq:][doc[N - Nq:] == d]
        total += int(np.searchsorted(mine, rows, side="right").sum())
    return total


def work(case):
    c = case
    B, N = c["batch"], c["tokens"]
    if c["op"] == "attn":
        H, Nq, kb = c["heads"], c["queries"] or N, c["key_block"]
        nk = (N + kb - 1) // kb
        share = sum(_budgets(c, nk)) / (nk * H)
        rows = B * H * Nq
        fixed = 2 * 64 * 2 * rows + 4 * rows + 2 * 64 * 2 * B * H * N
        lists = 4 * share * B * H * ((Nq + 127) // 128) * nk if c["keep"] < 1 else 0
        arrays = 4 * B * (N + Nq) * ((c["docs"] > 0) + (c["order"] != "none") + (c["bias"] != "none"))
        return {"bytes": fixed + lists + arrays, "flops": 4 * 64 * share * B * H * _pairs(c)}
    size = 4 if c["dtype"] == "fp32" else 2
    places = 4 * B * N * c["axes"]
    if c["op"] == "rope":
        n = B * c["heads"] * N
        return {"bytes": 2 * n * c["dim"] * size + places, "flops": 3 * n * c["rot"]}
    n = B * N * (c["heads"] + c["kv_heads"])
    moved = n + (B * N * c["kv_heads"] if c["with_v"] else 0)
    return {"bytes": 2 * moved * c["dim"] * size + places, "flops": n * (5 * c["dim"] + 3 * c["rot"])}


# ------------------------------------------------------------------------------- exact
def _exact_rotation(c, positions):
    """Complex factor e^{i angle} of every pair: [B, N, rot / 2], pairs in section order."""
    d = c["rot"] // c["axes"]
    theta = c["theta"] * (c["factor"] ** (d / (d - 2)) if c["scaling"] == "ntk" else 1.0)
    freq, amp = [], 1.0
    for i in range(d // 2):
        w = math.exp(-2.0 * i / d * math.log(theta))
        if c["scaling"] == "linear":
            w /= c["factor"]
        if c["scaling"] == "yarn":
            edge = [d * math.log(c["original"] / (r * 2 * math.pi)) / (2 * math.log(theta)) for r in (32.0, 1.0)]
            low, high = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), d - 1)
            mix = min(1.0, max(0.0, (i - low) / (high - low if high > low else 0.001)))
            w = w * (1 - mix) + w / c["factor"] * mix
        freq.append(w)
    if c["scaling"] == "yarn" and c["factor"] > 1:
        amp = 0.1 * math.log(c["factor"]) + 1
    f = torch.tensor(freq, dtype=torch.float64, device="cuda")
    ang = torch.cat([positions[..., a:a + 1].double() * f for a in range(c["axes"])], -1)
    return torch.polar(torch.full_like(ang, amp), ang)


def _exact_pairs(c):
    """Element numbers of the first and the second member of every pair."""
    d = c["rot"] // c["axes"]
    n = torch.arange(c["rot"] // 2, device="cuda")
    section, i = n // (d // 2), n % (d // 2)
    if c["layout"] == "half":
        return section * d + i, section * d + i + d // 2
    return section * d + 2 * i, section * d + 2 * i + 1


def _exact_turn(c, x, positions, inverse=False):
    """x [B, N, H, D] in 64 bits."""
    z = _exact_rotation(c, positions).unsqueeze(2)
    if inverse:
        z = z.conj()
    first, second = _exact_pairs(c)
    y = torch.complex(x[..., first], x[..., second]) * z
    out = x.clone()
    out[..., first] = y.real
    out[..., second] = y.imag
    return out


def _exact_attn(c, st):
    B, H, N, Nq, kb = c["batch"], c["heads"], c["tokens"], c["queries"] or c["tokens"], c["key_block"]
    out = torch.zeros(B, H, Nq, 64, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, Nq), -math.inf, dtype=torch.float64, device="cuda")
    nk = (N + kb - 1) // kb
    step = 2048                       # query rows at a time, whole query blocks
    block = torch.arange(N, device="cuda") // kb
    for b in range(B):
        for r0 in range(0, Nq, step):
            rows = slice(r0, min(Nq, r0 + step))
            n = rows.stop - rows.start
            hide = torch.zeros(n, N, dtype=torch.bool, device="cuda")
            if st["k_doc"] is not None:
                hide |= st["q_doc"][b, rows, None] != st["k_doc"][b]
                hide |= (st["k_doc"][b] < 0)
            if st["k_order"] is not None:
                hide |= st["k_order"][b] > st["q_order"][b, rows, None]
            for h in range(H):
                gone = hide
                if st["kv_idx"] is not None:
                    drop = torch.ones((n + 127) // 128, nk, dtype=torch.bool, device="cuda")
                    for i in range(drop.shape[0]):  # the row's list, in the words of its definition
                        row = r0 // 128 + i
                        drop[i, st["kv_idx"][b, h, row, :int(st["kv_cnt_host"][b, h, row])].long()] = False
                    gone = hide | drop[torch.arange(n, device="cuda") // 128][:, block]
                s = (st["q"][b, h, rows].double() @ st["k"][b, h].double().T) * st["scale"]
                if c["softcap"]:
                    s = torch.tanh(s / c["softcap"]).mul_(c["softcap"])
                if st["slopes"] is not None:
                    dist = (st["k_pos"][b].double() - st["q_pos"][b, rows, None].double()).abs()
                    s -= st["slopes"][h].double() * dist
                s.masked_fill_(gone, -math.inf)
                l = torch.logsumexp(s, -1)
                lse[b, h, rows] = l
                w = torch.exp(s - torch.where(torch.isinf(l), torch.zeros_like(l), l)[:, None])
                out[b, h, rows] = w @ st["v"][b, h].double()
    return {"out": out, "lse": lse}


def exact(case, seed):
    c, st = case, prepare(case, seed)
    if c["op"] == "attn":
        if st["kv_cnt"] is not None:
            st["kv_cnt_host"] = st["kv_cnt"].cpu()
        return _exact_attn(c, st)
    if c["op"] == "rope":
        y = _exact_turn(c, st["x"].double().transpose(1, 2), st["positions"], c["inverse"])
        return y.transpose(1, 2)
    H, G = c["heads"], c["kv_heads"]
    B, N, T = c["batch"], c["tokens"], c["tokens"] // c["views"]
    x = st["packed"].double()
    t = torch.arange(N, device="cuda")
    v, r = t // T, t % T
    patch = T - c["specials"]
    to = torch.where(r >= c["specials"], v * patch + r - c["specials"], c["views"] * patch + v * c["specials"] + r)
    result = {}
    for n, y in (("q", x[:, :, :H]), ("k", x[:, :, H:H + G]), ("v", x[:, :, H + G:])):
        if n == "v" and not c["with_v"]:
            continue
        if n != "v":
            if c["norm"] == "layer":
                y = (y - y.mean(-1, keepdim=True)) / torch.sqrt(y.var(-1, unbiased=False, keepdim=True) + 1e-5)
            else:
                y = y / torch.sqrt(y.pow(2).mean(-1, keepdim=True) + 1e-5)
            if st[n + "_weight"] is not None:
                y = y * st[n + "_weight"].double()
            if st[n + "_bias"] is not None:
                y = y + st[n + "_bias"].double()
            y = _exact_turn(c, y, st["positions"])
        moved = torch.empty_like(y)
        moved[:, to] = y
        result[n] = moved.transpose(1, 2)
    return result
