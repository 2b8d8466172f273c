"""Oracle of the token operators and of attention with changed scores, in 64 bits.

TEST INFRASTRUCTURE, as ress_oracle.py: imported by the tests only, imports nothing from the
product.  Plain restatements of the definitions in include/ress.h; torch float64 on the
device of the inputs, so that layer-sized cases stay quick.
"""
from __future__ import annotations

import math

import torch


def frequencies(d: int, theta: float, scaling: str = "none", factor: float = 1.0, original_len: int = 0,
                beta_fast: float = 32.0, beta_slow: float = 1.0):
    """Radians per position of the d/2 pairs of a section of d elements, and the amplitude."""
    if scaling == "ntk":
        theta = theta * factor ** (d / (d - 2))
    f = [theta ** (-2.0 * i / d) for i in range(d // 2)]
    if scaling == "linear":
        f = [x / factor for x in f]
    if scaling != "yarn":
        return f, 1.0
    edge = [d * math.log(original_len / (n * 2 * math.pi)) / (2 * math.log(theta)) for n in (beta_fast, beta_slow)]
    low, high = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), d - 1)
    ramp = [min(1.0, max(0.0, (i - low) / max(high - low, 0.001))) for i in range(d // 2)]
    return [x / factor * r + x * (1 - r) for x, r in zip(f, ramp)], 0.1 * math.log(factor) + 1


def pair_elements(rot: int, axes: int, layout: str):
    """(first, second, axis, pair-of-section) of every rotated pair."""
    d = rot // axes
    out = []
    for a in range(axes):
        for i in range(d // 2):
            base = a * d
            e = (base + i, base + i + d // 2) if layout == "half" else (base + 2 * i, base + 2 * i + 1)
            out.append((*e, a, i))
    return out


def rope(x, positions, rot, axes, layout, freq, amplitude, inverse=False):
    """x [B, H, N, D] float64; positions [B, N, axes] (integers)."""
    y = x.clone()
    f = torch.tensor(freq, dtype=torch.float64, device=x.device)
    for e0, e1, a, i in pair_elements(rot, axes, layout):
        w = (positions[:, :, a].double() * f[i]).unsqueeze(1)
        c, s = amplitude * torch.cos(w), amplitude * torch.sin(w) * (-1 if inverse else 1)
        y[..., e0] = x[..., e0] * c - x[..., e1] * s
        y[..., e1] = x[..., e1] * c + x[..., e0] * s
    return y


def head_norm(x, norm: str, eps: float, weight=None, bias=None):
    """x [B, H, N, D] float64.  Returns the normalised rows and their factor 1 / sqrt(...)."""
    if norm == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    if norm == "none":
        return x, torch.ones_like(r)
    y = x * r
    if weight is not None:
        y = y * weight.double()
    return (y if bias is None else y + bias.double()), r


def tail_order(tokens: int, views: int, specials: int):
    """Place of every token in the order of ress_token_gather."""
    T = tokens // views
    out = []
    for t in range(tokens):
        v, w = divmod(t, T)
        out.append(views * (T - specials) + v * specials + w if w < specials else v * (T - specials) + w - specials)
    return out


def masked_attn(q, k, v, scale, key_block=128, kv_lists=None, softcap=0.0, slopes=None, q_pos=None, k_pos=None,
                q_doc=None, k_doc=None, q_order=None, k_order=None):
    """Attention with changed scores, row by row of the definition, in float64.  q [B,H,Nq,64],
    k, v [B,H,N,64] (any type); kv_lists {(b, h, i): [key blocks]} or None.  Returns out, lse,
    sum_u w_u |v_u| and max_u sum_i |q_i k_i| scale over the seen keys (for error bounds)."""
    B, H, Nq, D = q.shape
    N = k.shape[2]
    dev = q.device
    out = torch.zeros(B, H, Nq, D, dtype=torch.float64, device=dev)
    size = torch.zeros_like(out)
    lse = torch.full((B, H, Nq), -math.inf, dtype=torch.float64, device=dev)
    reach = torch.zeros(B, H, Nq, dtype=torch.float64, device=dev)
    if N == 0:
        return out, lse, size, reach
    nk = (N + key_block - 1) // key_block
    for b in range(B):
        seen = torch.ones(Nq, N, dtype=torch.bool, device=dev)
        if q_doc is not None:
            seen &= (q_doc[b][:, None] == k_doc[b][None, :]) & (q_doc[b][:, None] >= 0)
        if q_order is not None:
            seen &= k_order[b][None, :] <= q_order[b][:, None]
        for h in range(H):
            times = torch.ones(Nq, N, dtype=torch.float64, device=dev)
            if kv_lists is not None:
                times.zero_()
                for i in range((Nq + 127) // 128):
                    n = torch.zeros(nk, dtype=torch.float64, device=dev)
                    for j in kv_lists[(b, h, i)]:
                        n[j] += 1
                    times[128 * i:128 * i + 128] = n.repeat_interleave(key_block)[:N]
            vis = seen & (times > 0)
            # a hidden key is dropped before any arithmetic: what it holds does not matter
            any_ = vis.any(0)
            kk = torch.where(any_[:, None], k[b, h].double(), torch.zeros(D, dtype=torch.float64, device=dev))
            s = q[b, h].double() @ kk.T * scale
            if softcap:
                s = softcap * torch.tanh(s / softcap)
            if slopes is not None:
                s = s - slopes[h].double() * (q_pos[b].double()[:, None] - k_pos[b].double()[None, :]).abs()
            s = torch.where(vis, s + torch.log(times), torch.full_like(s, -math.inf))
            m = s.amax(-1, keepdim=True)
            m = torch.where(m == -math.inf, torch.zeros_like(m), m)
            w = torch.exp(s - m)
            l = w.sum(-1, keepdim=True)
            lse[b, h] = (m + torch.log(l)).squeeze(-1)
            w = torch.where(l > 0, w / l, torch.zeros_like(w))
            vv = v[b, h].double()
            fin = torch.isfinite(vv).all(-1)
            ok = torch.where(fin[:, None], vv, torch.zeros_like(vv))
            out[b, h] = w @ ok
            size[b, h] = w @ ok.abs()
            for u in torch.nonzero(~fin & any_).flatten().tolist():
                rows = vis[:, u]
                out[b, h, rows] += w[rows, u, None] * vv[u]
                size[b, h, rows] += w[rows, u, None] * vv[u].abs()
            reach[b, h] = torch.where(vis, q[b, h].double().abs() @ kk.abs().T * scale, torch.zeros_like(s)).amax(-1)
    return out, lse, size, reach
