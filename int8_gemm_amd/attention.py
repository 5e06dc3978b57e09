"""Rotary tables, norms of queries and keys, and attention: the binding of the
convrot_rope_table, convrot_qk_norm_rope and convrot_attention entry points
(include/convrot.h has the definitions). Checks, streams and errors are those of
the rest of the binding."""

from __future__ import annotations

import ctypes
import math

import torch

from . import _DTYPES, load_library
from .mx4 import _NORMS, _U8, _launch, _tensor

__all__ = ["convrot_rope_table", "convrot_qk_norm_rope", "convrot_attention",
           "convrot_attention_workspace_size"]

_POSITIONS = {torch.int32: 0, torch.int64: 1, torch.float32: 2}
_I32 = torch.int32


class _QkArgs(ctypes.Structure):
    _fields_ = ([(f, ctypes.c_void_p) for f in ("q", "k", "q_out", "k_out", "q_weight",
                                                "k_weight", "table")]
                + [(f, ctypes.c_int64) for f in (
                    "q_stride", "q_head_stride", "k_stride", "k_head_stride", "q_out_stride",
                    "q_out_head_stride", "k_out_stride", "k_out_head_stride", "tokens",
                    "table_rows")]
                + [(f, ctypes.c_int32) for f in ("q_heads", "k_heads", "d", "pairs")]
                + [("norm", ctypes.c_int), ("row", ctypes.c_int32), ("halves", ctypes.c_int32),
                   ("dtype", ctypes.c_int), ("eps", ctypes.c_float)])


class _AttentionArgs(ctypes.Structure):
    _fields_ = ([(f, ctypes.c_void_p) for f in ("q", "k", "v", "out", "lse", "q_offsets",
                                                "k_offsets", "k_lens")]
                + [(f, ctypes.c_int64) for f in (
                    "q_stride", "q_head_stride", "k_stride", "k_head_stride", "v_stride",
                    "v_head_stride", "out_stride", "out_head_stride", "q_tokens", "k_tokens",
                    "batch")]
                + [(f, ctypes.c_int32) for f in ("q_heads", "k_heads", "d", "causal")]
                + [("dtype", ctypes.c_int), ("scale", ctypes.c_float)])


def _heads(t, name: str, dtype, dev: int):
    """Check a [tokens, heads, d] or [batch, length, heads, d] tensor; (address,
    tokens, heads, d, token stride, head stride, batch)."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype:
        raise TypeError(f"{name} must be a {dtype} tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected device {dev}")
    shape, strides = t.shape, t.stride()
    batch = 1
    if len(shape) == 4:
        batch, length, heads, d = shape
        tokens = batch * length
        # sequences follow one another at the tokens' stride
        if batch > 1 and length > 1 and strides[0] != length * strides[1]:
            raise ValueError(f"{name}: its sequences do not follow one another (shape "
                             f"{tuple(shape)}, strides {strides})")
        stride = strides[1] if length > 1 else strides[0]
    elif len(shape) == 3:
        tokens, heads, d = shape
        stride = strides[0]
    else:
        raise ValueError(f"{name} must be [tokens, heads, d] or [batch, length, heads, d] "
                         f"(got shape {tuple(shape)})")
    if strides[-1] != 1 and d > 1 and t.numel():
        raise ValueError(f"{name}: the elements of a head must be consecutive (strides {strides})")
    # strides that nothing steps over say nothing
    if tokens <= 1:
        stride = (heads * d + 7) // 8 * 8
    return (t.data_ptr(), tokens, heads, d, stride, strides[-2] if heads > 1 else (d + 7) // 8 * 8,
            batch)


def _first(t, name: str) -> int:
    """Check the tensor that the others have to fit; its device index."""
    if not isinstance(t, torch.Tensor) or t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be a bfloat16 or float16 tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a ROCm device (got {t.device})")
    return t.get_device()


def convrot_rope_table(positions: torch.Tensor, dims, theta: float = 10000.0, *,
                       shared: bool = False, out: torch.Tensor | None = None):
    """cos and sin of the angles of `positions` [tokens, axes] (or [tokens]: one
    axis; int32, int64 or float32) as fp32 [tokens, pairs, 2]. Axis a turns
    dims[a] / 2 pairs; `shared`: one ladder of frequencies over all axes."""
    if not isinstance(positions, torch.Tensor) or positions.dtype not in _POSITIONS:
        raise TypeError("positions must be an int32, int64 or float32 tensor")
    if not positions.is_cuda:
        raise ValueError(f"positions must be on a ROCm device (got {positions.device})")
    dims = tuple(int(n) for n in dims)
    if positions.dim() == 1 and len(dims) == 1:
        axis_stride = 0
    elif positions.dim() == 2 and positions.shape[1] == len(dims):
        axis_stride = positions.stride(1)
    else:
        raise ValueError(f"positions of shape {tuple(positions.shape)} do not fit {len(dims)} axes")
    tokens, dev = positions.shape[0], positions.get_device()
    pairs = sum(dims) // 2
    if out is None:
        out = torch.empty((tokens, pairs, 2), dtype=torch.float32, device=positions.device)
        po = out.data_ptr()
    else:
        po = _tensor(out, "out", torch.float32, (tokens, pairs, 2), dev)
    _launch("convrot_rope_table", dev, positions.data_ptr(), _POSITIONS[positions.dtype],
            positions.stride(0), axis_stride, tokens, len(dims),
            (ctypes.c_int32 * max(1, len(dims)))(*dims), theta, int(shared), po)
    return out


def convrot_qk_norm_rope(q: torch.Tensor, k: torch.Tensor | None = None,
                         table: torch.Tensor | None = None, *, norm: str | None = "rms",
                         span: str = "head", q_weight: torch.Tensor | None = None,
                         k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                         halves: bool = False, q_out: torch.Tensor | None = None,
                         k_out: torch.Tensor | None = None):
    """Norms of q and k ('rms', 'layer' or None) over each head or, span='row',
    over all heads of a token, and the rotation of `table` [rows, pairs, 2] (rows
    dividing the tokens), in one pass. q, k [tokens, heads, d] or [batch, length,
    heads, d] bf16 or fp16, of any strides with consecutive heads' elements;
    weights [d] or [heads * d]. Returns (q', k'), k' None without k; `q_out=q`
    works in place."""
    if norm not in _NORMS or span not in ("head", "row"):
        raise ValueError(f"norm={norm!r}, span={span!r}: 'rms', 'layer' or None; 'head' or 'row'")
    dev, dtype = _first(q, "q"), q.dtype
    a = _QkArgs(norm=_NORMS[norm], row=span == "row", halves=halves, dtype=_DTYPES[dtype], eps=eps)
    a.q, tokens, heads, d, a.q_stride, a.q_head_stride, _ = _heads(q, "q", dtype, dev)
    a.tokens, a.q_heads, a.d = tokens, heads, d
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=dtype, device=q.device)
    elif q_out.shape != q.shape:
        raise ValueError(f"q_out must have shape {tuple(q.shape)} (got {tuple(q_out.shape)})")
    a.q_out, _, _, _, a.q_out_stride, a.q_out_head_stride, _ = _heads(q_out, "q_out", dtype, dev)
    if q_weight is not None:
        a.q_weight = _weight(q_weight, "q_weight", dtype, dev, d, heads if span == "row" else 1)
    if k is not None:
        a.k, k_tokens, a.k_heads, k_d, a.k_stride, a.k_head_stride, _ = _heads(k, "k", dtype, dev)
        if k_tokens != tokens or k_d != d:
            raise ValueError(f"k {tuple(k.shape)} does not fit q {tuple(q.shape)}")
        if k_out is None:
            k_out = torch.empty(k.shape, dtype=dtype, device=k.device)
        elif k_out.shape != k.shape:
            raise ValueError(f"k_out must have shape {tuple(k.shape)} (got {tuple(k_out.shape)})")
        a.k_out, _, _, _, a.k_out_stride, a.k_out_head_stride, _ = _heads(k_out, "k_out", dtype,
                                                                         dev)
        if k_weight is not None:
            a.k_weight = _weight(k_weight, "k_weight", dtype, dev, d,
                                 a.k_heads if span == "row" else 1)
    elif k_weight is not None or k_out is not None:
        raise ValueError("k_weight and k_out need k")
    if table is not None:
        if table.dim() != 3 or table.shape[2] != 2:
            raise ValueError(f"table must be [rows, pairs, 2] (got shape {tuple(table.shape)})")
        a.table = _tensor(table, "table", torch.float32, tuple(table.shape), dev)
        a.table_rows, a.pairs = table.shape[0], table.shape[1]
    _launch("convrot_qk_norm_rope", dev, ctypes.byref(a))
    return q_out, k_out


def _weight(t, name: str, dtype, dev: int, d: int, heads: int) -> int:
    shape = (heads * d,) if heads == 1 or t.dim() == 1 else (heads, d)
    return _tensor(t, name, dtype, shape, dev)


def _attention_args(q, k, v, q_offsets, k_offsets, k_lens, causal, scale):
    dev, dtype = _first(q, "q"), q.dtype
    a = _AttentionArgs(causal=causal, dtype=_DTYPES[dtype])
    a.q, a.q_tokens, a.q_heads, d, a.q_stride, a.q_head_stride, q_batch = _heads(q, "q", dtype, dev)
    a.k, k_tokens, k_heads, k_d, a.k_stride, a.k_head_stride, k_batch = _heads(k, "k", dtype, dev)
    a.v, v_tokens, v_heads, v_d, a.v_stride, a.v_head_stride, _ = _heads(v, "v", dtype, dev)
    if (k_tokens, k_heads, k_d) != (v_tokens, v_heads, v_d) or k_d != d:
        raise ValueError(f"q {tuple(q.shape)}, k {tuple(k.shape)} and v {tuple(v.shape)} do not "
                         "fit")
    a.k_tokens, a.k_heads, a.d = k_tokens, k_heads, d
    batch = None
    for t, name, of, n in ((q_offsets, "q_offsets", q, q_batch), (k_offsets, "k_offsets", k,
                                                                  k_batch)):
        if t is not None:
            n = t.numel() - 1
            setattr(a, name, _tensor(t, name, _I32, (n + 1,), dev))
            if of.dim() == 4:
                raise ValueError(f"{name} need a packed [tokens, heads, d] tensor")
        if batch is not None and n != batch:
            raise ValueError(f"{batch} sequences of queries, {n} of keys")
        batch = n
    if batch < 1:
        raise ValueError("offsets have one entry more than there are sequences")
    a.batch = batch
    if k_lens is not None:
        a.k_lens = _tensor(k_lens, "k_lens", _I32, (batch,), dev)
    a.scale = 1.0 / math.sqrt(d) if scale is None else scale
    return a, dev


def convrot_attention_workspace_size(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *,
                                     q_offsets: torch.Tensor | None = None,
                                     k_offsets: torch.Tensor | None = None) -> int:
    """Workspace bytes of a convrot_attention call with these tensors."""
    a, _ = _attention_args(q, k, v, q_offsets, k_offsets, None, False, None)
    return int(load_library().convrot_attention_workspace_size(ctypes.byref(a)))


def convrot_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *,
                      q_offsets: torch.Tensor | None = None,
                      k_offsets: torch.Tensor | None = None,
                      k_lens: torch.Tensor | None = None, causal: bool = False,
                      scale: float | None = None, return_lse: bool = False,
                      out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None):
    """softmax(scale q k^T) v per sequence and head; out like q, and lse
    [q_heads, tokens] fp32 where `return_lse` or `lse` ask for it.

    q [tokens, q_heads, d], k, v [tokens, k_heads, d] bf16 or fp16 packed by
    `q_offsets` and `k_offsets` (int32 [batch + 1]; none: one sequence), or
    [batch, length, heads, d]; k_lens (int32 [batch]): the keys in use of each
    sequence. `causal` masks lower right. Rows that no sequence owns are not
    written. `workspace` (uint8 on the device) defaults to what the call asks for."""
    a, dev = _attention_args(q, k, v, q_offsets, k_offsets, k_lens, causal, scale)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    elif out.shape != q.shape:
        raise ValueError(f"out must have shape {tuple(q.shape)} (got {tuple(out.shape)})")
    a.out, _, _, _, a.out_stride, a.out_head_stride, _ = _heads(out, "out", q.dtype, dev)
    if lse is not None:
        a.lse = _tensor(lse, "lse", torch.float32, (a.q_heads, a.q_tokens), dev)
    elif return_lse:
        lse = torch.empty((a.q_heads, a.q_tokens), dtype=torch.float32, device=q.device)
        a.lse = lse.data_ptr()
    if workspace is None:
        size = load_library().convrot_attention_workspace_size(ctypes.byref(a))
        if size:
            workspace = torch.empty_strided((size,), (1,), dtype=_U8, device=q.device)
            pw = workspace.data_ptr()
        else:
            pw = None
    else:
        pw = _tensor(workspace, "workspace", _U8, (workspace.numel(),), dev)
        size = workspace.numel()
    _launch("convrot_attention", dev, ctypes.byref(a), pw, size)
    return out if lse is None else (out, lse)
