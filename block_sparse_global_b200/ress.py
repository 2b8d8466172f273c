"""ctypes binding of libress.so: the C entry points of include/ress.h under the same names.

Argument marshalling only: shapes and parameters are packed into the C structs, torch
tensors are passed as raw device pointers, and a non-OK status raises RessError.  Every
step of the computation runs in the library's CUDA kernels.  If libress.so has not been
built, the first call raises RessError (there is no fallback implementation).
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading
from typing import Optional, Sequence

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libress.so")

RESS_OK = 0
STATUS_NAMES = {0: "RESS_OK", 1: "RESS_ERR_INVALID_ARG", 2: "RESS_ERR_UNSUPPORTED",
                3: "RESS_ERR_CUDA", 4: "RESS_ERR_DEVICE_BOUNDS", 5: "RESS_ERR_DEVICE_TIMEOUT"}
SELECT_MASS, SELECT_DRIFT, SELECT_RANDOM, SELECT_CDF = 0, 1, 2, 3
DRIFT_MINIMISE, DRIFT_MAXIMISE_SWAPS, DRIFT_MAXIMISE_FULL = 0, 1, 2
HEAD_DIM, BLOCK = 64, 128
MAX_TOKEN_DIM = 256
DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}
NORM_NONE, NORM_RMS, NORM_LAYER = 0, 1, 2


class RessError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {STATUS_NAMES.get(status, status)}")
        self.status = status


class ress_shape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("heads", ctypes.c_int32), ("seq_len", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("block", ctypes.c_int32),
                ("key_block", ctypes.c_int32)]


class ress_select_params(ctypes.Structure):
    _fields_ = [("method", ctypes.c_int32), ("budgets", ctypes.POINTER(ctypes.c_int32)),
                ("keep_k", ctypes.c_void_p), ("dense_q", ctypes.c_void_p),
                ("rounds", ctypes.c_int32), ("rho", ctypes.c_float), ("eps", ctypes.c_float),
                ("seed", ctypes.c_uint64), ("objective", ctypes.c_int32), ("top_p", ctypes.c_float),
                ("drift", ctypes.c_void_p)]


class ress_rope_plan(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int32), ("rot_dim", ctypes.c_int32), ("axes", ctypes.c_int32),
                ("layout", ctypes.c_int32), ("amplitude", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("phase", ctypes.c_uint64 * (MAX_TOKEN_DIM // 2))]


class ress_rows(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("stride_b", ctypes.c_int64),
                ("stride_h", ctypes.c_int64), ("stride_t", ctypes.c_int64)]


class ress_qk_params(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("tokens", ctypes.c_int32), ("q_heads", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("norm", ctypes.c_int32), ("eps", ctypes.c_float),
                ("q_weight", ctypes.c_void_p), ("q_bias", ctypes.c_void_p),
                ("k_weight", ctypes.c_void_p), ("k_bias", ctypes.c_void_p),
                ("rope", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("pos_stride_b", ctypes.c_int64), ("views", ctypes.c_int32),
                ("specials", ctypes.c_int32)]


class ress_attn_mods(ctypes.Structure):
    _fields_ = [("q_len", ctypes.c_int32), ("softcap", ctypes.c_float)] + [
        (n, ctypes.c_void_p) for n in ("slopes", "q_pos", "k_pos", "q_doc", "k_doc", "q_order",
                                       "k_order")]


_lib = None
_lock = threading.Lock()
_VP, _I32, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
_SIGS = {
    "ress_abi_version": (_I32, []),
    "ress_status_string": (ctypes.c_char_p, [_I32]),
    "ress_head_gram": (_I32, [ctypes.POINTER(ress_shape), _I32, _VP, _VP, _VP]),
    "ress_token_gather": (_I32, [ctypes.POINTER(ress_shape), _I32, _I32, _I32, _VP, _VP, _VP]),
    "ress_pool_blocks": (_I32, [ctypes.POINTER(ress_shape), _VP, _VP, _VP, _VP, _VP, _VP, _VP]),
    "ress_block_scores": (_I32, [ctypes.POINTER(ress_shape), _VP, _VP, _VP, ctypes.c_float, _VP,
                                 _VP, _VP]),
    "ress_drift_workspace_bytes": (_SZ, [ctypes.POINTER(ress_shape)]),
    "ress_drift_scores": (_I32, [ctypes.POINTER(ress_shape), _VP, _VP, _VP, _VP, _VP, _VP, _SZ,
                                 _VP]),
    "ress_drift_scores_static": (_I32, [ctypes.POINTER(ress_shape), _VP, _VP, _VP, _VP, _VP, _VP]),
    "ress_select_blocks": (_I32, [ctypes.POINTER(ress_shape), ctypes.POINTER(ress_select_params),
                                  _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP]),
    "ress_scores_select": (_I32, [ctypes.POINTER(ress_shape), ctypes.POINTER(ress_select_params),
                                  _VP, _VP, _VP, ctypes.c_float, _VP, _VP, _VP, _VP, _VP, _VP,
                                  _VP]),
    "ress_drift_select_workspace_bytes": (_SZ, [ctypes.POINTER(ress_shape)]),
    "ress_drift_select": (_I32, [ctypes.POINTER(ress_shape), ctypes.POINTER(ress_select_params),
                                 _VP, _VP, _VP, _VP, ctypes.c_float, _VP, _VP, _VP, _VP, _VP,
                                 _VP, _VP, _VP, _SZ, _VP]),
    "ress_attn_schedule": (_I32, [ctypes.POINTER(ress_shape), _VP, _VP, _VP]),
    "ress_block_sparse_attn": (_I32, [ctypes.POINTER(ress_shape), _VP, _VP, _VP, _VP, _VP, _VP,
                                      ctypes.c_float, _VP, _VP, _VP, _VP]),
    "ress_debug_attn_forced_timeout": (_I32, [ctypes.POINTER(ress_shape), _VP, _VP, _VP, _VP,
                                              _VP, ctypes.c_float, _VP, _VP, ctypes.c_int64,
                                              _VP]),
    "ress_masked_attn_workspace_bytes": (_SZ, [ctypes.POINTER(ress_shape), _I32]),
    "ress_masked_attn": (_I32, [ctypes.POINTER(ress_shape), ctypes.POINTER(ress_attn_mods), _VP,
                                _VP, _VP, _VP, _VP, _VP, ctypes.c_float, _VP, _VP, _VP, _SZ, _VP,
                                _VP]),
    "ress_rope_init": (_I32, [ctypes.POINTER(ress_rope_plan), _I32, _I32, _I32, _I32,
                              ctypes.c_double, _I32, ctypes.c_double, _I32, ctypes.c_double,
                              ctypes.c_double]),
    "ress_rope": (_I32, [ctypes.POINTER(ress_rope_plan), _I32, _I32, _I32, _I32,
                         ctypes.POINTER(ress_rows), _VP, ctypes.c_int64, _I32,
                         ctypes.POINTER(ress_rows), _VP]),
    "ress_qk_norm_rope": (_I32, [_VP] * 8),
}


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Loads libress.so (once).  Raises RessError-compatible RuntimeError if missing."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise RuntimeError(f"libress.so not built at {path}; run "
                                   "`python -m block_sparse_global_b200.build`")
            lib = ctypes.CDLL(path)
            for name, (res, args) in _SIGS.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
        return _lib


def _check(fn: str, status: int):
    if status != RESS_OK:
        raise RessError(fn, status)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor or None")
    if not t.is_contiguous():
        raise ValueError("tensors passed to libress must be contiguous")
    return t.data_ptr() or None


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def make_shape(batch: int, heads: int, seq_len: int, head_dim: int = HEAD_DIM,
               block: int = BLOCK, key_block: int = 0) -> ress_shape:
    """key_block 0 means key blocks of the query block's size (128); 64 is the grid of
    ReSS Supp. F (128-token query blocks, 64-token key blocks)."""
    return ress_shape(batch, heads, seq_len, head_dim, block, key_block)


def grid(seq_len: int, key_block: int = 0):
    """(nq, nk): query blocks of 128 tokens and key blocks of key_block tokens."""
    kb = key_block or BLOCK
    return (seq_len + BLOCK - 1) // BLOCK, (seq_len + kb - 1) // kb


def _shape(shape) -> ress_shape:
    if isinstance(shape, ress_shape):
        return shape
    return make_shape(*shape)


def ress_abi_version() -> int:
    return load().ress_abi_version()


def ress_status_string(status: int) -> str:
    return load().ress_status_string(status).decode()


def ress_head_gram(shape, w_o: torch.Tensor, gram: torch.Tensor, stream=None):
    st = load().ress_head_gram(ctypes.byref(_shape(shape)), int(w_o.shape[0]), _ptr(w_o),
                               _ptr(gram), _stream(stream))
    _check("ress_head_gram", st)


def ress_pool_blocks(shape, q, k, v, q_pool, k_pool, v_pool, stream=None):
    st = load().ress_pool_blocks(ctypes.byref(_shape(shape)), _ptr(q), _ptr(k), _ptr(v),
                                 _ptr(q_pool), _ptr(k_pool), _ptr(v_pool), _stream(stream))
    _check("ress_pool_blocks", st)


def ress_block_scores(shape, q_pool, k_pool, v_pool, scale: float, P, v_bar, stream=None):
    st = load().ress_block_scores(ctypes.byref(_shape(shape)), _ptr(q_pool), _ptr(k_pool),
                                  _ptr(v_pool), float(scale), _ptr(P), _ptr(v_bar), _stream(stream))
    _check("ress_block_scores", st)


def ress_drift_workspace_bytes(shape) -> int:
    return int(load().ress_drift_workspace_bytes(ctypes.byref(_shape(shape))))


def ress_drift_scores(shape, P, v_pool, v_bar, gram, s, workspace: torch.Tensor, stream=None):
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = load().ress_drift_scores(ctypes.byref(_shape(shape)), _ptr(P), _ptr(v_pool), _ptr(v_bar),
                                  _ptr(gram), _ptr(s), _ptr(workspace), nbytes, _stream(stream))
    _check("ress_drift_scores", st)


def ress_drift_scores_static(shape, P, v_pool, v_bar, gram, s, stream=None):
    """Drift score with the library's fixed static scratch (no workspace argument), for
    callers that cannot allocate device memory; see include/ress.h."""
    st = load().ress_drift_scores_static(ctypes.byref(_shape(shape)), _ptr(P), _ptr(v_pool),
                                         _ptr(v_bar), _ptr(gram), _ptr(s), _stream(stream))
    _check("ress_drift_scores_static", st)


def select_params(method: int, budgets: Sequence[int], keep_k=None, dense_q=None, rounds: int = 0,
                  rho: float = 0.5, eps: float = 1e-4, seed: int = 0, objective: int = 0,
                  drift=None, top_p: float = 1.0):
    """Packs ress_select_params (`drift`: optional fp32 [B,H,nb] device tensor for the
    realized J per row).  Returns (struct, host budget array that must stay alive)."""
    arr = (ctypes.c_int32 * len(budgets))(*[int(b) for b in budgets])
    p = ress_select_params(int(method), ctypes.cast(arr, ctypes.POINTER(ctypes.c_int32)),
                           _ptr(keep_k), _ptr(dense_q), int(rounds), float(rho), float(eps),
                           int(seed) & ((1 << 64) - 1), int(objective), float(top_p), _ptr(drift))
    return p, arr


def ress_select_blocks(shape, params, P, s, v_pool, v_bar, gram, kv_idx, kv_cnt, mask=None,
                       dev_err=None, stream=None):
    """params: a ress_select_params, or the (struct, budgets) pair of select_params()."""
    keep = None
    if isinstance(params, tuple):
        params, keep = params
    st = load().ress_select_blocks(ctypes.byref(_shape(shape)), ctypes.byref(params), _ptr(P),
                                   _ptr(s), _ptr(v_pool), _ptr(v_bar), _ptr(gram), _ptr(kv_idx),
                                   _ptr(kv_cnt), _ptr(mask), _ptr(dev_err), _stream(stream))
    del keep
    _check("ress_select_blocks", st)


def ress_scores_select(shape, params, q_pool, k_pool, v_pool, scale: float, P, v_bar, kv_idx,
                       kv_cnt, mask=None, dev_err=None, stream=None):
    """Block map fused with MASS / RANDOM selection; P and v_bar may be None."""
    keep = None
    if isinstance(params, tuple):
        params, keep = params
    st = load().ress_scores_select(ctypes.byref(_shape(shape)), ctypes.byref(params), _ptr(q_pool),
                                   _ptr(k_pool), _ptr(v_pool), float(scale), _ptr(P), _ptr(v_bar),
                                   _ptr(kv_idx), _ptr(kv_cnt), _ptr(mask), _ptr(dev_err),
                                   _stream(stream))
    del keep
    _check("ress_scores_select", st)


def ress_drift_select_workspace_bytes(shape) -> int:
    return int(load().ress_drift_select_workspace_bytes(ctypes.byref(_shape(shape))))


def ress_drift_select(shape, params, q_pool, k_pool, v_pool, gram, scale: float, P, v_bar, s,
                      kv_idx, kv_cnt, workspace: torch.Tensor, mask=None, dev_err=None,
                      stream=None):
    """Block map, drift score and DRIFT selection in one kernel; P, v_bar, s may be None."""
    keep = None
    if isinstance(params, tuple):
        params, keep = params
    st = load().ress_drift_select(ctypes.byref(_shape(shape)), ctypes.byref(params), _ptr(q_pool),
                                  _ptr(k_pool), _ptr(v_pool), _ptr(gram), float(scale), _ptr(P),
                                  _ptr(v_bar), _ptr(s), _ptr(kv_idx), _ptr(kv_cnt), _ptr(mask),
                                  _ptr(dev_err), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _stream(stream))
    del keep
    _check("ress_drift_select", st)


def ress_token_gather(shape, views: int, specials: int, inverse: bool, src, dst, stream=None):
    """Moves every view's special tokens to the tail (inverse=False) or back."""
    st = load().ress_token_gather(ctypes.byref(_shape(shape)), int(views), int(specials),
                                  1 if inverse else 0, _ptr(src), _ptr(dst), _stream(stream))
    _check("ress_token_gather", st)


def ress_attn_schedule(shape, kv_cnt, work_order, stream=None):
    st = load().ress_attn_schedule(ctypes.byref(_shape(shape)), _ptr(kv_cnt), _ptr(work_order),
                                   _stream(stream))
    _check("ress_attn_schedule", st)


def ress_block_sparse_attn(shape, q, k, v, kv_idx, kv_cnt, work_order, scale: float, out,
                           lse=None, dev_err=None, stream=None):
    st = load().ress_block_sparse_attn(ctypes.byref(_shape(shape)), _ptr(q), _ptr(k), _ptr(v),
                                       _ptr(kv_idx), _ptr(kv_cnt), _ptr(work_order), float(scale),
                                       _ptr(out), _ptr(lse), _ptr(dev_err), _stream(stream))
    _check("ress_block_sparse_attn", st)


def ress_debug_attn_forced_timeout(shape, q, k, v, kv_idx, kv_cnt, scale: float, out, dev_err,
                                   limit_cycles: int, stream=None):
    """Diagnostics of the device error path (see include/ress.h): the attention kernel with
    every CTA's softmax stalled on a barrier that nothing completes, so that each takes its
    bounded-wait timeout path and writes RESS_ERR_DEVICE_TIMEOUT to dev_err."""
    st = load().ress_debug_attn_forced_timeout(ctypes.byref(_shape(shape)), _ptr(q), _ptr(k),
                                               _ptr(v), _ptr(kv_idx), _ptr(kv_cnt), float(scale),
                                               _ptr(out), _ptr(dev_err), int(limit_cycles),
                                               _stream(stream))
    _check("ress_debug_attn_forced_timeout", st)


# ------------------------------------------------------------------- token operators
def rope_plan(head_dim: int, rot_dim: Optional[int] = None, axes: int = 1, layout: str = "half",
              theta: float = 10000.0, scaling: str = "none", factor: float = 1.0,
              original_len: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """The rotation of a model (ress_rope_init): computed once, passed to every call.
    rot_dim: leading elements that are rotated (default: all of head_dim); layout "half" or
    "interleaved"; scaling "none", "linear", "ntk" or "yarn"."""
    if layout not in ROPE_LAYOUTS or scaling not in ROPE_SCALINGS:
        raise ValueError(f"unknown rotary layout {layout!r} or scaling {scaling!r}")
    plan = ress_rope_plan()
    st = load().ress_rope_init(ctypes.byref(plan), int(head_dim),
                               int(head_dim if rot_dim is None else rot_dim), int(axes),
                               ROPE_LAYOUTS[layout], float(theta), ROPE_SCALINGS[scaling],
                               float(factor), int(original_len), float(beta_fast),
                               float(beta_slow))
    _check("ress_rope_init", st)
    return plan


def _rows(t: torch.Tensor, shape, dtype, device):
    """A [B, heads, N, D] tensor of this shape, type and device as the fields of ress_rows."""
    if t.shape != shape or t.dtype != dtype or t.device != device:
        raise ValueError(f"expected {dtype} {tuple(shape)} on {device}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    b, h, n, e = t.stride()
    if e != 1 and shape[3] > 1:
        raise ValueError("the elements of a row must be contiguous")
    return t.data_ptr(), b, h, n


def _positions(plan, positions, batch: int, tokens: int, device):
    """(pointer, batch stride) of int32 positions [tokens], [tokens, axes], [batch or 1, tokens]
    or [batch or 1, tokens, axes]."""
    if positions is None:
        return None, 0
    if positions.dtype != torch.int32 or positions.device != device:
        raise ValueError("positions must be int32 on the tensors' device")
    axes = plan.axes
    p = positions
    if p.dim() == 3 and p.shape == (batch, tokens, axes) and p.is_contiguous():
        return p.data_ptr() or None, tokens * axes
    if axes == 1 and p.dim() <= 2 and (p.dim() == 1 or p.shape[-1] == tokens and p.shape[0] in (1, batch)):
        p = p.unsqueeze(-1)
    if p.dim() == 2:
        p = p.unsqueeze(0)
    if p.dim() != 3 or p.shape[1:] != (tokens, axes) or p.shape[0] not in (1, batch):
        raise ValueError(f"positions of shape {tuple(positions.shape)} do not fit "
                         f"{batch} x {tokens} tokens and {axes} axes")
    if (axes > 1 and p.stride(2) != 1) or (tokens > 1 and p.stride(1) != axes):
        raise ValueError("the positions of a batch entry must be contiguous")
    return p.data_ptr() or None, (p.stride(0) if p.shape[0] > 1 else 0)


def _launch(name: str, device, stream, *args):
    """Calls the library with the tensors' device current, on `stream` or that device's current
    stream."""
    if device.type != "cuda":
        raise ValueError(f"{name} takes CUDA tensors, got {device}")
    if stream is None:  # (the same stream as torch.cuda.current_stream, without its lookups)
        stream = torch._C._cuda_getCurrentRawStream(device.index)
    elif isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            st = getattr(load(), name)(*args, int(stream))
    else:
        st = getattr(_lib or load(), name)(*args, int(stream))
    _check(name, st)


def ress_rope(plan, x: torch.Tensor, positions: Optional[torch.Tensor], out: torch.Tensor,
              inverse: bool = False, stream=None):
    """Rotates x [B, heads, N, D] (any strides over whole rows) into out (may be x)."""
    shape, dtype, dev = x.shape, x.dtype, x.device
    if len(shape) != 4 or shape[3] != plan.head_dim or dtype not in DTYPES:
        raise ValueError(f"expected [B, heads, N, {plan.head_dim}] of bf16, fp16 or fp32")
    src, dst = ress_rows(*_rows(x, shape, dtype, dev)), ress_rows(*_rows(out, shape, dtype, dev))
    b, h, n, _ = shape
    pos, pos_b = _positions(plan, positions, b, n, dev)
    _launch("ress_rope", dev, stream, plan, b, h, n, DTYPES[dtype], src, pos, pos_b,
            1 if inverse else 0, dst)


class _QkBlock(ctypes.Structure):
    _fields_ = [("params", ress_qk_params), ("rows", ress_rows * 6)]


_QK_PACK = struct.Struct("=7if6Qq2i" + "Q3q" * 6)
_QK_ROWS_AT = _QkBlock.rows.offset
assert _QK_PACK.size == ctypes.sizeof(_QkBlock) and ctypes.sizeof(ress_rows) == 32


def _affine(w: Optional[torch.Tensor], dim: int, device):
    if w is None:
        return 0
    if w.dtype != torch.float32 or w.shape != (dim,) or w.device != device or not w.is_contiguous():
        raise ValueError(f"norm weights and biases must be fp32 [{dim}] on the tensors' device")
    return w.data_ptr()


def ress_qk_norm_rope(q, k, q_out, k_out, v=None, v_out=None, norm: int = NORM_RMS,
                      eps: float = 1e-6, q_weight=None, q_bias=None, k_weight=None, k_bias=None,
                      plan=None, positions=None, views: int = 1, specials: int = 0, stream=None):
    """Per-head norm and rotation of q and k (and the move of v) in one pass, into the token
    order of ress_token_gather.  Tensors are [B, heads, N, D] views of any strides."""
    shape, dtype, dev = q.shape, q.dtype, q.device
    if len(shape) != 4 or k.dim() != 4 or dtype not in DTYPES:
        raise ValueError("expected [batch, heads, tokens, head_dim] tensors of bf16, fp16 or fp32")
    if (v is None) != (v_out is None):
        raise ValueError("v and v_out go together")
    b, h, n, d = shape
    kv = k.shape
    if kv[0] != b or kv[2] != n or kv[3] != d:
        raise ValueError(f"q {tuple(shape)} and k {tuple(kv)} do not belong together")
    pos, pos_b = (None, 0) if plan is None else _positions(plan, positions, b, n, dev)
    none = (0, 0, 0, 0)
    block = _QkBlock()  # the structs of the call, filled at once
    _QK_PACK.pack_into(
        block, 0, b, n, h, kv[1], d, DTYPES[dtype], norm, eps, _affine(q_weight, d, dev),
        _affine(q_bias, d, dev), _affine(k_weight, d, dev), _affine(k_bias, d, dev),
        0 if plan is None else ctypes.addressof(plan), pos or 0, pos_b, views, specials,
        *_rows(q, shape, dtype, dev), *_rows(k, kv, dtype, dev),
        *(none if v is None else _rows(v, kv, dtype, dev)), *_rows(q_out, shape, dtype, dev),
        *_rows(k_out, kv, dtype, dev), *(none if v is None else _rows(v_out, kv, dtype, dev)))
    at = ctypes.addressof(block)
    q_at = at + _QK_ROWS_AT
    _launch("ress_qk_norm_rope", dev, stream, at, q_at, q_at + 32, None if v is None else q_at + 64,
            q_at + 96, q_at + 128, None if v is None else q_at + 160)


# ------------------------------------------------------- attention with changed scores
def ress_masked_attn_workspace_bytes(shape, q_len: int) -> int:
    return int(load().ress_masked_attn_workspace_bytes(ctypes.byref(_shape(shape)), int(q_len)))


def _sized(t: Optional[torch.Tensor], shape, dtype, device, name: str):
    """Device pointer of a contiguous tensor of exactly this shape, type and device, or None."""
    if t is None:
        return None
    if t.shape != shape or t.dtype != dtype or t.device != device:
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)} on {device}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr() or None


def ress_masked_attn(shape, q, k, v, kv_idx, kv_cnt, work_order, scale: float, out, lse=None,
                     softcap: float = 0.0, slopes=None, q_pos=None, k_pos=None, q_doc=None,
                     k_doc=None, q_order=None, k_order=None, workspace=None, dev_err=None,
                     stream=None):
    """Attention over kept blocks with capped scores, a distance bias and document and order
    masks, for all tokens or for others: q [B,H,q_len,64] over k, v [B,H,N,64].  kv_idx and
    kv_cnt None: every key block.  `workspace`: uint8, ress_masked_attn_workspace_bytes (None
    where that is 0)."""
    s = _shape(shape)
    dev = q.device
    if q.dim() != 4:
        raise ValueError("expected q [B, H, q_len, 64]")
    B, H, N, n = s.batch, s.heads, s.seq_len, q.shape[2]
    nq, nk = grid(n)[0], grid(N, s.key_block)[1]
    bf, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    qd, kd = (B, n), (B, N)
    m = ress_attn_mods(n, softcap)
    if slopes is not None:
        m.slopes = _sized(slopes, (H,), f32, dev, "slopes")
    if q_pos is not None or k_pos is not None:
        m.q_pos, m.k_pos = _sized(q_pos, qd, i32, dev, "q_pos"), _sized(k_pos, kd, i32, dev, "k_pos")
    if q_doc is not None or k_doc is not None:
        m.q_doc, m.k_doc = _sized(q_doc, qd, i32, dev, "q_doc"), _sized(k_doc, kd, i32, dev, "k_doc")
    if q_order is not None or k_order is not None:
        m.q_order = _sized(q_order, qd, i32, dev, "q_order")
        m.k_order = _sized(k_order, kd, i32, dev, "k_order")
    nbytes = 0
    if workspace is not None:
        if workspace.device != dev:
            raise ValueError("the workspace is on another device")
        nbytes = workspace.numel() * workspace.element_size()
    if work_order is not None and (work_order.numel() != B * H * nq or work_order.dtype != i32
                                   or work_order.device != dev):
        raise ValueError("work_order holds one int32 entry per row")
    if dev_err is not None and (dev_err.dtype != i32 or dev_err.device != dev):
        raise ValueError("dev_err is an int32 word on the tensors' device")
    rows, keys = (B, H, n, 64), (B, H, N, 64)
    _launch("ress_masked_attn", dev, stream, s, m, _sized(q, rows, bf, dev, "q"),
            _sized(k, keys, bf, dev, "k"), _sized(v, keys, bf, dev, "v"),
            None if kv_idx is None else _sized(kv_idx, (B, H, nq, nk), i32, dev, "kv_idx"),
            None if kv_cnt is None else _sized(kv_cnt, (B, H, nq), i32, dev, "kv_cnt"),
            None if work_order is None else _ptr(work_order), scale,
            _sized(out, rows, bf, dev, "out"), _sized(lse, (B, H, n), f32, dev, "lse"),
            _ptr(workspace), nbytes, None if dev_err is None else _ptr(dev_err))
