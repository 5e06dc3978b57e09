"""Rotary tables, norms of queries and keys, and attention: the binding of the
convrot_rope_table, convrot_qk_norm_rope and convrot_attention entry points
(include/convrot.h has the definitions). Checks, streams and errors are those of
the rest of the binding."""

from __future__ import annotations

import ctypes
import struct

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


_pack_qk = struct.Struct("@7Q10q8if4x").pack  # a _QkArgs at a third of its host time


class _AttentionArgs(ctypes.Structure):
    _fields_ = ([(f, ctypes.c_void_p) for f in ("q", "k", "v", "out", "lse", "q_offsets",
                                                "k_offsets", "k_lens")]
                + [(f, ctypes.c_int64) for f in (
                    "q_stride", "q_head_stride", "k_stride", "k_head_stride", "v_stride",
                    "v_head_stride", "out_stride", "out_head_stride", "q_tokens", "k_tokens",
                    "batch")]
                + [(f, ctypes.c_int32) for f in ("q_heads", "k_heads", "d", "causal")]
                + [("dtype", ctypes.c_int), ("scale", ctypes.c_float), ("tile", ctypes.c_int32)])


_pack_attention = struct.Struct("@8Q11q5ifi4x").pack
_OUT, _LSE, _OUT_STRIDE, _OUT_HEAD_STRIDE, _TOKENS = 3, 4, 14, 15, 16  # of its fields

# As in mx4.py: one expression on the good path, what is wrong is worked out behind it.

def _heads(t, name: str, dtype, dev: int):
    """Check a [tokens, heads, d] or [batch, length, heads, d] tensor; (address,
    tokens, heads, d, token stride, head stride, batch)."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev:
        shape, strides = t.shape, t.stride()
        if len(shape) == 3 and strides[2] == 1:
            tokens, heads, d = shape
            if tokens > 1 and heads > 1:
                return t.data_ptr(), tokens, heads, d, strides[0], strides[1], 1
    elif not isinstance(t, torch.Tensor) or t.dtype is not dtype:
        raise TypeError(f"{name} must be a {dtype} tensor")
    else:
        raise ValueError(f"{name} is on {t.device}, expected device {dev}")
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


def _like(x: torch.Tensor, tokens: int, heads: int, d: int):
    """A new contiguous tensor of x's shape; with its address and strides as _heads'."""
    if x.is_contiguous():
        out = torch.empty_like(x)  # a fifth less host time
        return out, out.data_ptr(), heads * d, d
    out = torch.empty_strided(x.shape, (heads * d, d, 1) if x.dim() == 3 else
                              (tokens // x.shape[0] * heads * d if x.shape[0] else 1, heads * d,
                               d, 1), dtype=x.dtype, device=x.device)
    return out, out.data_ptr(), heads * d, d


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
        out = torch.empty_strided((tokens, pairs, 2), (2 * pairs, 2, 1), dtype=torch.float32,
                                  device=positions.device)
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
    dev, dtype, row = _first(q, "q"), q.dtype, span == "row"
    pq, tokens, heads, d, qs, qh, _ = _heads(q, "q", dtype, dev)
    if q_out is None:
        q_out, pqo, qos, qoh = _like(q, tokens, heads, d)
    elif q_out is q:
        pqo, qos, qoh = pq, qs, qh
    else:
        pqo, qos, qoh = _output(q_out, "q_out", q, dev)
    pqw = 0 if q_weight is None else _weight(q_weight, "q_weight", dtype, dev, d,
                                                heads if row else 1)
    pk = pko = pkw = 0
    k_heads = ks = kh = kos = koh = 0
    if k is not None:
        pk, k_tokens, k_heads, k_d, ks, kh, _ = _heads(k, "k", dtype, dev)
        if k_tokens != tokens or k_d != d:
            raise ValueError(f"k {tuple(k.shape)} does not fit q {tuple(q.shape)}")
        if k_out is None:
            k_out, pko, kos, koh = _like(k, tokens, k_heads, d)
        elif k_out is k:
            pko, kos, koh = pk, ks, kh
        else:
            pko, kos, koh = _output(k_out, "k_out", k, dev)
        if k_weight is not None:
            pkw = _weight(k_weight, "k_weight", dtype, dev, d, k_heads if row else 1)
    elif k_weight is not None or k_out is not None:
        raise ValueError("k_weight and k_out need k")
    pt, rows, pairs = 0, 0, 0
    if table is not None:
        shape = table.shape if isinstance(table, torch.Tensor) else ()
        if len(shape) != 3 or shape[2] != 2:
            raise ValueError(f"table must be [rows, pairs, 2] (got shape {tuple(shape)})")
        pt = _tensor(table, "table", torch.float32, shape, dev)
        rows, pairs, _ = shape
    a = _pack_qk(pq, pk, pqo, pko, pqw, pkw, pt, qs, qh, ks, kh, qos, qoh, kos, koh, tokens, rows,
                 heads, k_heads, d, pairs, _NORMS[norm], row, halves, _DTYPES[dtype], eps)
    _launch("convrot_qk_norm_rope", dev, a)
    return q_out, k_out


def _output(out, name: str, like: torch.Tensor, dev: int):
    """Check an output of another tensor's shape; (address, token and head stride)."""
    p, _, _, _, stride, head_stride, _ = _heads(out, name, like.dtype, dev)
    if out.shape != like.shape:
        raise ValueError(f"{name} must have shape {tuple(like.shape)} (got {tuple(out.shape)})")
    return p, stride, head_stride


def _weight(t, name: str, dtype, dev: int, d: int, heads: int) -> int:
    flat = heads == 1 or not isinstance(t, torch.Tensor) or t.dim() == 1
    shape = (heads * d,) if flat else (heads, d)
    return _tensor(t, name, dtype, shape, dev)


def _sequences(offsets, name: str, of: torch.Tensor, batch: int, dev: int):
    """Check offsets into `of`, whose own batch counts without them; (address, sequences)."""
    if offsets is None:
        return 0, batch
    n = offsets.numel() - 1 if isinstance(offsets, torch.Tensor) else 0
    p = _tensor(offsets, name, _I32, (n + 1,), dev)
    if of.dim() == 4:
        raise ValueError(f"{name} need a packed [tokens, heads, d] tensor")
    if n < 1:
        raise ValueError(f"{name} have one entry more than there are sequences")
    return p, n


def _attention_args(q, k, v, q_offsets, k_offsets, k_lens, causal, scale, tile):
    """The fields of _AttentionArgs but the outputs', and the device index."""
    dev, dtype = _first(q, "q"), q.dtype
    pq, tokens, heads, d, qs, qh, batch = _heads(q, "q", dtype, dev)
    pk, k_tokens, k_heads, k_d, ks, kh, k_batch = _heads(k, "k", dtype, dev)
    pv, v_tokens, v_heads, v_d, vs, vh, _ = _heads(v, "v", dtype, dev)
    if k_tokens != v_tokens or k_heads != v_heads or k_d != d or v_d != d:
        raise ValueError(f"q {tuple(q.shape)}, k {tuple(k.shape)} and v {tuple(v.shape)} do not "
                         "fit")
    pqo, batch = _sequences(q_offsets, "q_offsets", q, batch, dev)
    pko, k_batch = _sequences(k_offsets, "k_offsets", k, k_batch, dev)
    if batch != k_batch:
        raise ValueError(f"{batch} sequences of queries, {k_batch} of keys")
    pkl = 0 if k_lens is None else _tensor(k_lens, "k_lens", _I32, (batch,), dev)
    return [pq, pk, pv, 0, 0, pqo, pko, pkl, qs, qh, ks, kh, vs, vh, 0, 0, tokens, k_tokens, batch,
            heads, k_heads, d, causal, _DTYPES[dtype],
            max(d, 1) ** -0.5 if scale is None else scale, tile], dev


def convrot_attention_workspace_size(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *,
                                     q_offsets: torch.Tensor | None = None,
                                     k_offsets: torch.Tensor | None = None,
                                     causal: bool = False, tile: int = 0) -> int:
    """Workspace bytes of a convrot_attention call with these tensors."""
    a, _ = _attention_args(q, k, v, q_offsets, k_offsets, None, causal, None, tile)
    return int(load_library().convrot_attention_workspace_size(_pack_attention(*a)))


def convrot_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *,
                      q_offsets: torch.Tensor | None = None,
                      k_offsets: torch.Tensor | None = None,
                      k_lens: torch.Tensor | None = None, causal: bool = False,
                      scale: float | None = None, return_lse: bool = False,
                      out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, tile: int = 0):
    """softmax(scale q k^T) v per sequence and head; out like q, and lse
    [q_heads, tokens] fp32 where `return_lse` or `lse` ask for it.

    q [tokens, q_heads, d], k, v [tokens, k_heads, d] bf16 or fp16 packed by
    `q_offsets` and `k_offsets` (int32 [batch + 1]; none: one sequence), or
    [batch, length, heads, d]; k_lens (int32 [batch]): the keys in use of each
    sequence. `causal` masks lower right; `scale` defaults to d^-1/2. Rows that no
    sequence owns are not written. `workspace` (uint8 on the device) defaults to what
    the call asks for. `tile` != 0 forces a kernel (test / tuning hook)."""
    a, dev = _attention_args(q, k, v, q_offsets, k_offsets, k_lens, causal, scale, tile)
    heads, d = q.shape[-2:]
    tokens = a[_TOKENS]
    if out is None:
        out, a[_OUT], a[_OUT_STRIDE], a[_OUT_HEAD_STRIDE] = _like(q, tokens, heads, d)
    else:
        a[_OUT], a[_OUT_STRIDE], a[_OUT_HEAD_STRIDE] = _output(out, "out", q, dev)
    if lse is not None:
        a[_LSE] = _tensor(lse, "lse", torch.float32, (heads, tokens), dev)
    elif return_lse:
        lse = torch.empty_strided((heads, tokens), (tokens, 1), dtype=torch.float32,
                                  device=q.device)
        a[_LSE] = lse.data_ptr()
    a = _pack_attention(*a)
    pw, size = None, 0
    if workspace is not None:
        size = workspace.numel() if isinstance(workspace, torch.Tensor) else 0
        pw = _tensor(workspace, "workspace", _U8, (size,), dev)
    else:
        size = load_library().convrot_attention_workspace_size(a)
        if size:
            workspace = torch.empty_strided((size,), (1,), dtype=_U8, device=q.device)
            pw = workspace.data_ptr()
    _launch("convrot_attention", dev, a, pw, size)
    return out if lse is None else (out, lse)
