"""Microscaled 4-bit (MXFP4) layers and the gated residual norm: the binding of
the convrot_*_mx4 and convrot_norm_residual entry points (include/convrot.h has
the format and the numerics). Like the rest of the binding it checks torch
tensors, passes pointers and the tensors' current stream, and raises
ConvrotError on a non-OK status; shapes of every buffer are checked here."""

from __future__ import annotations

import ctypes

import torch

from . import _DTYPES, ROT_SEED, _check, load_library

__all__ = [
    "convrot_quantize_mx4", "convrot_dequant_mx4", "convrot_gemm_mx4", "convrot_linear_mx4",
    "convrot_linear_mx4_workspace_size", "convrot_linear_mx4_workspace_for_rows",
    "convrot_mx4_scales_size", "convrot_norm_residual", "convrot_norm_residual_mx4",
]

_NORMS = {None: 0, "rms": 1, "layer": 2}


class _NormArgs(ctypes.Structure):
    _fields_ = ([(f, ctypes.c_void_p) for f in ("x", "o", "x_out", "post_weight", "weight",
                                                "gate", "scale", "shift")]
                + [(f, ctypes.c_int64) for f in ("gate_stride", "scale_stride", "shift_stride")]
                + [(f, ctypes.c_void_p) for f in ("h", "h_codes", "h_scales")]
                + [(f, ctypes.c_int64) for f in ("m", "k", "rows_per_mod")]
                + [("rot_seed", ctypes.c_uint64), ("post_norm", ctypes.c_int),
                   ("norm", ctypes.c_int), ("dtype", ctypes.c_int), ("g", ctypes.c_int32),
                   ("eps", ctypes.c_float)])


def _tensor(t, name: str, dtype: torch.dtype, shape: tuple, device: torch.device) -> int:
    """Check a tensor (dtype, shape, contiguity, device); its address."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape} (got {tuple(t.shape)})")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _input16(x, name: str) -> int:
    """Check a 2-D bf16 / half input on a device; its convrot_dtype."""
    if not isinstance(x, torch.Tensor) or x.dtype not in _DTYPES:
        raise TypeError(f"{name} must be a bfloat16 or float16 tensor")
    if not x.is_cuda:
        raise ValueError(f"{name} must be on a ROCm device (got {x.device})")
    if x.dim() != 2:
        raise ValueError(f"{name} must be 2-D (got shape {tuple(x.shape)})")
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return _DTYPES[x.dtype]


def _dtype16(dtype) -> int:
    if dtype not in _DTYPES:
        raise TypeError("dtype must be torch.bfloat16 or torch.float16")
    return _DTYPES[dtype]


def _scales_shape(rows: int, k: int) -> tuple:
    return (-(-k // 256), -(-rows // 16) * 16, 8)


def _quantized(codes, scales, name: str):
    """Check a quantized tensor; (rows, k, codes address, scales address)."""
    if not isinstance(codes, torch.Tensor) or codes.dim() != 2:
        raise TypeError(f"{name} codes must be a 2-D uint8 tensor")
    if not codes.is_cuda:
        raise ValueError(f"{name} codes must be on a ROCm device (got {codes.device})")
    rows, half = codes.shape
    dev = codes.device
    return (rows, 2 * half, _tensor(codes, f"{name} codes", torch.uint8, (rows, half), dev),
            _tensor(scales, f"{name} scales", torch.uint8, _scales_shape(rows, 2 * half), dev))


def _new_quantized(rows: int, k: int, dev, codes, scales):
    """The output pair of a quantization, allocated where not given."""
    if codes is None:
        codes = torch.empty((rows, k // 2), dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty(_scales_shape(rows, k), dtype=torch.uint8, device=dev)
    return (codes, scales, _tensor(codes, "codes", torch.uint8, (rows, k // 2), dev),
            _tensor(scales, "scales", torch.uint8, _scales_shape(rows, k), dev))


def _launch(fn, dev: torch.device, *args) -> None:
    """Call an entry point on `dev`'s current stream (with `dev` current)."""
    stream = torch.cuda.current_stream(dev).cuda_stream
    if torch.cuda.current_device() == dev.index:
        _check(fn(*args, stream))
    else:
        with torch.cuda.device(dev):
            _check(fn(*args, stream))


def convrot_mx4_scales_size(rows: int, k: int) -> int:
    """Bytes of the scales tensor of a quantized [rows, k] tensor."""
    return int(load_library().convrot_mx4_scales_size(rows, k))


def convrot_quantize_mx4(x: torch.Tensor, g: int, rot_seed: int = ROT_SEED, *,
                         codes: torch.Tensor | None = None, scales: torch.Tensor | None = None):
    """x [rows, k] bf16 or fp16 (weight or activations) -> (codes uint8
    [rows, k/2], scales uint8 [ceil(k/256), rows rounded up to 16, 8]), rotated
    in groups of g (1: not rotated)."""
    dt = _input16(x, "x")
    rows, k = x.shape
    codes, scales, pc, ps = _new_quantized(rows, k, x.device, codes, scales)
    _launch(load_library().convrot_quantize_mx4, x.device, x.data_ptr(), dt, rows, k, g, rot_seed,
            pc, ps)
    return codes, scales


def convrot_dequant_mx4(codes: torch.Tensor, scales: torch.Tensor, g: int,
                        rot_seed: int = ROT_SEED, *, dtype: torch.dtype = torch.bfloat16,
                        out: torch.Tensor | None = None):
    """The [rows, k] tensor in `dtype` that codes and scales stand for, rotated
    back in groups of g (1: the values as they are held)."""
    dt = _dtype16(dtype)
    rows, k, pc, ps = _quantized(codes, scales, "")
    dev = codes.device
    out = torch.empty((rows, k), dtype=dtype, device=dev) if out is None else out
    _launch(load_library().convrot_dequant_mx4, dev, pc, ps, rows, k, g, rot_seed,
            _tensor(out, "out", dtype, (rows, k), dev), dt)
    return out


def convrot_gemm_mx4(x_codes: torch.Tensor, x_scales: torch.Tensor, w_codes: torch.Tensor,
                     w_scales: torch.Tensor, bias: torch.Tensor | None = None, *,
                     dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
                     tile: int = 0):
    """y [m, n] = x . w^T (+ bias) in `dtype` over two quantized tensors. `tile`
    != 0 forces a kernel variant (test / tuning hook)."""
    dt = _dtype16(dtype)
    m, k, xc, xs = _quantized(x_codes, x_scales, "x")
    n, kw, wc, ws = _quantized(w_codes, w_scales, "w")
    dev = x_codes.device
    if kw != k:
        raise ValueError(f"K mismatch: x has {k}, w has {kw}")
    if w_codes.device != dev:
        raise ValueError(f"x is on {dev}, w on {w_codes.device}")
    pb = None if bias is None else _tensor(bias, "bias", dtype, (n,), dev)
    out = torch.empty((m, n), dtype=dtype, device=dev) if out is None else out
    _launch(load_library().convrot_gemm_mx4, dev, xc, xs, wc, ws, pb, m, n, k,
            _tensor(out, "out", dtype, (m, n), dev), dt, tile)
    return out


def convrot_linear_mx4_workspace_for_rows(rows: int, k: int) -> int:
    return int(load_library().convrot_linear_mx4_workspace_for_rows(rows, k))


def convrot_linear_mx4_workspace_size(m: int, n: int, k: int) -> int:
    return int(load_library().convrot_linear_mx4_workspace_size(m, n, k))


def convrot_linear_mx4(x: torch.Tensor, w_codes: torch.Tensor, w_scales: torch.Tensor, g: int,
                       rot_seed: int = ROT_SEED, bias: torch.Tensor | None = None, *,
                       workspace: torch.Tensor | None = None, out: torch.Tensor | None = None):
    """The forward of a layer whose weight convrot_quantize_mx4 made with the
    same g and rot_seed: x [m, k] bf16 or fp16 -> y [m, n] in x's format.
    `workspace` (uint8 on the device) defaults to the library's default size."""
    dt = _input16(x, "x")
    m, k = x.shape
    dev = x.device
    n, kw, wc, ws = _quantized(w_codes, w_scales, "w")
    if kw != k:
        raise ValueError(f"K mismatch: x has {k}, w has {kw}")
    if w_codes.device != dev:
        raise ValueError(f"x is on {dev}, w on {w_codes.device}")
    pb = None if bias is None else _tensor(bias, "bias", x.dtype, (n,), dev)
    lib = load_library()
    if workspace is None:
        workspace = torch.empty(lib.convrot_linear_mx4_workspace_size(m, n, k),
                                dtype=torch.uint8, device=dev)
    pw = _tensor(workspace, "workspace", torch.uint8, tuple(workspace.shape), dev)
    out = torch.empty((m, n), dtype=x.dtype, device=dev) if out is None else out
    _launch(lib.convrot_linear_mx4, dev, x.data_ptr(), wc, ws, pb, m, n, k, g, rot_seed,
            _tensor(out, "out", x.dtype, (m, n), dev), dt, pw, workspace.numel())
    return out


def _modulation(t, name: str, x: torch.Tensor, samples: int):
    """Check a modulation ([k] or [b, k], rows of any stride); (address, stride, b)."""
    if t is None:
        return None, 0, samples
    k = x.shape[1]
    if not isinstance(t, torch.Tensor) or t.dtype != x.dtype:
        raise TypeError(f"{name} must be a {x.dtype} tensor")
    if t.device != x.device:
        raise ValueError(f"{name} is on {t.device}, expected {x.device}")
    if t.dim() not in (1, 2) or t.shape[-1] != k or t.stride(-1) != 1:
        raise ValueError(f"{name} must be [{k}] or [samples, {k}] with contiguous rows "
                         f"(got shape {tuple(t.shape)}, strides {t.stride()})")
    if t.dim() == 1 or t.shape[0] == 1:
        return t.data_ptr(), 0, samples
    if samples not in (0, t.shape[0]):
        raise ValueError(f"{name} has {t.shape[0]} samples, another modulation {samples}")
    if t.shape[0] == 0 or x.shape[0] % t.shape[0]:
        raise ValueError(f"{x.shape[0]} rows do not divide into {t.shape[0]} samples")
    return t.data_ptr(), t.stride(0), t.shape[0]


def _norm_args(x, o, gate, post_norm, post_weight, norm, weight, scale, shift, eps, x_out):
    dt = _input16(x, "x")
    m, k = x.shape
    dev, dtype = x.device, x.dtype
    if norm not in ("rms", "layer") or post_norm not in _NORMS:
        raise ValueError(f"norm={norm!r}, post_norm={post_norm!r}: 'rms' or 'layer'")
    a = _NormArgs(x=x.data_ptr(), m=m, k=k, dtype=dt, norm=_NORMS[norm],
                  post_norm=_NORMS[post_norm], eps=eps)
    if o is not None:
        a.o = _tensor(o, "o", dtype, (m, k), dev)
        x_out = torch.empty((m, k), dtype=dtype, device=dev) if x_out is None else x_out
        a.x_out = _tensor(x_out, "x_out", dtype, (m, k), dev)
    elif x_out is not None or gate is not None or post_norm is not None:
        raise ValueError("x_out, gate and post_norm need o")
    else:
        x_out = x
    if post_weight is not None:
        a.post_weight = _tensor(post_weight, "post_weight", dtype, (k,), dev)
    if weight is not None:
        a.weight = _tensor(weight, "weight", dtype, (k,), dev)
    samples = 0
    a.gate, a.gate_stride, samples = _modulation(gate, "gate", x, samples)
    a.scale, a.scale_stride, samples = _modulation(scale, "scale", x, samples)
    a.shift, a.shift_stride, samples = _modulation(shift, "shift", x, samples)
    a.rows_per_mod = max(1, m // samples if samples else m)
    return a, x_out


def convrot_norm_residual(x: torch.Tensor, o: torch.Tensor | None = None, *,
                          gate: torch.Tensor | None = None, post_norm: str | None = None,
                          post_weight: torch.Tensor | None = None, norm: str = "rms",
                          weight: torch.Tensor | None = None, scale: torch.Tensor | None = None,
                          shift: torch.Tensor | None = None, eps: float = 1e-6,
                          x_out: torch.Tensor | None = None, h: torch.Tensor | None = None):
    """x' = x + gate * post_norm(o); h = norm(x') * (1 + scale) + shift.

    x, o [m, k] bf16 or fp16; weights [k]; gate, scale, shift [k] or
    [samples, k] (rows of any stride: column ranges of one projection do), a
    sample's rows of x being consecutive. Returns (x', h); x' is x where o is
    None. `x_out=x` updates x in place."""
    a, x_out = _norm_args(x, o, gate, post_norm, post_weight, norm, weight, scale, shift, eps,
                          x_out)
    h = torch.empty_like(x) if h is None else h
    a.h = _tensor(h, "h", x.dtype, tuple(x.shape), x.device)
    _launch(load_library().convrot_norm_residual, x.device, ctypes.byref(a))
    return x_out, h


def convrot_norm_residual_mx4(x: torch.Tensor, o: torch.Tensor | None, g: int,
                              rot_seed: int = ROT_SEED, *, gate: torch.Tensor | None = None,
                              post_norm: str | None = None,
                              post_weight: torch.Tensor | None = None, norm: str = "rms",
                              weight: torch.Tensor | None = None,
                              scale: torch.Tensor | None = None,
                              shift: torch.Tensor | None = None, eps: float = 1e-6,
                              x_out: torch.Tensor | None = None, h: torch.Tensor | None = None,
                              codes: torch.Tensor | None = None,
                              scales: torch.Tensor | None = None):
    """convrot_norm_residual with h rotated in groups of g and quantized for
    convrot_gemm_mx4: returns (x', codes, scales), the same bits as
    convrot_quantize_mx4 of the 16-bit h. `h`, where given, is written too."""
    a, x_out = _norm_args(x, o, gate, post_norm, post_weight, norm, weight, scale, shift, eps,
                          x_out)
    codes, scales, a.h_codes, a.h_scales = _new_quantized(*x.shape, x.device, codes, scales)
    a.g, a.rot_seed = g, rot_seed
    if h is not None:
        a.h = _tensor(h, "h", x.dtype, tuple(x.shape), x.device)
    _launch(load_library().convrot_norm_residual, x.device, ctypes.byref(a))
    return x_out, codes, scales
