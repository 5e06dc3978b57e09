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

# the address of a device's current stream, without the Stream object around it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda dev: torch.cuda.current_stream(dev).cuda_stream)
# no initialisation check: the callers hold device tensors
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)

_U8 = torch.uint8
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


# A small call lasts about as long on the GPU as its checks here, so each check
# is one expression on the good path and works out what is wrong behind it.

def _tensor(t, name: str, dtype: torch.dtype, shape: tuple, dev: int) -> int:
    """Check a tensor (dtype, shape, contiguity, device index); its address."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.get_device() == dev and t.is_contiguous()):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape} (got {tuple(t.shape)})")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected device {dev}")
    raise ValueError(f"{name} must be contiguous")


def _input16(x, name: str) -> int:
    """Check a 2-D bf16 / half input on a device; its convrot_dtype."""
    if not isinstance(x, torch.Tensor) or x.dtype not in _DTYPES:
        raise TypeError(f"{name} must be a bfloat16 or float16 tensor")
    if x.is_cuda and x.dim() == 2 and x.is_contiguous():
        return _DTYPES[x.dtype]
    if not x.is_cuda:
        raise ValueError(f"{name} must be on a ROCm device (got {x.device})")
    if x.dim() != 2:
        raise ValueError(f"{name} must be 2-D (got shape {tuple(x.shape)})")
    raise ValueError(f"{name} must be contiguous")


def _dtype16(dtype) -> int:
    if dtype not in _DTYPES:
        raise TypeError("dtype must be torch.bfloat16 or torch.float16")
    return _DTYPES[dtype]


def _scales_shape(rows: int, k: int) -> tuple:
    return ((k + 255) // 256, (rows + 15) // 16 * 16, 8)


def _quantized(codes, scales, name: str):
    """Check a quantized tensor; (rows, k, codes address, scales address, device index)."""
    if (isinstance(codes, torch.Tensor) and codes.dtype is _U8 and codes.dim() == 2
            and codes.is_cuda and codes.is_contiguous()):
        rows, half = codes.shape
        dev = codes.get_device()
        return (rows, 2 * half, codes.data_ptr(),
                _tensor(scales, name + "scales", _U8, _scales_shape(rows, 2 * half), dev), dev)
    if not isinstance(codes, torch.Tensor) or codes.dim() != 2 or codes.dtype != _U8:
        raise TypeError(f"{name}codes must be a 2-D uint8 tensor")
    if not codes.is_cuda:
        raise ValueError(f"{name}codes must be on a ROCm device (got {codes.device})")
    raise ValueError(f"{name}codes must be contiguous")


def _empty(rows: int, cols: int, dtype: torch.dtype, device: torch.device) -> torch.Tensor:
    """torch.empty((rows, cols)) at a quarter less host time."""
    return torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=device)


def _new_quantized(rows: int, k: int, x: torch.Tensor, codes, scales):
    """The output pair of a quantization of `x`, allocated where not given; with
    its addresses."""
    cs, ss = (rows, k // 2), _scales_shape(rows, k)
    if codes is None:
        codes = _empty(rows, k // 2, _U8, x.device)
        pc = codes.data_ptr()
    else:
        pc = _tensor(codes, "codes", _U8, cs, x.get_device())
    if scales is None:
        scales = torch.empty_strided(ss, (8 * ss[1], 8, 1), dtype=_U8, device=x.device)
        ps = scales.data_ptr()
    else:
        ps = _tensor(scales, "scales", _U8, ss, x.get_device())
    return codes, scales, pc, ps


def _output(out, name: str, shape: tuple, dtype: torch.dtype, like: torch.Tensor):
    """The output `out`, allocated beside `like` where it is None; with its address."""
    if out is None:
        out = _empty(*shape, dtype, like.device)
        return out, out.data_ptr()
    return out, _tensor(out, name, dtype, shape, like.get_device())


_entry = {}  # entry points by name, bound at their first call


def _launch(name: str, dev: int, *args) -> None:
    """Call an entry point on device `dev`'s current stream (with `dev` current)."""
    fn = _entry.get(name)
    if fn is None:
        fn = _entry[name] = getattr(load_library(), name)
    if _current_device() != dev:
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(dev))
    else:
        status = fn(*args, _raw_stream(dev))
    if status:
        _check(status)


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
    codes, scales, pc, ps = _new_quantized(rows, k, x, codes, scales)
    _launch("convrot_quantize_mx4", x.get_device(), x.data_ptr(), dt, rows, k, g, rot_seed, pc, ps)
    return codes, scales


def convrot_dequant_mx4(codes: torch.Tensor, scales: torch.Tensor, g: int,
                        rot_seed: int = ROT_SEED, *, dtype: torch.dtype = torch.bfloat16,
                        out: torch.Tensor | None = None):
    """The [rows, k] tensor in `dtype` that codes and scales stand for, rotated
    back in groups of g (1: the values as they are held)."""
    dt = _dtype16(dtype)
    rows, k, pc, ps, dev = _quantized(codes, scales, "")
    out, po = _output(out, "out", (rows, k), dtype, codes)
    _launch("convrot_dequant_mx4", dev, pc, ps, rows, k, g, rot_seed, po, dt)
    return out


def convrot_gemm_mx4(x_codes: torch.Tensor, x_scales: torch.Tensor, w_codes: torch.Tensor,
                     w_scales: torch.Tensor, bias: torch.Tensor | None = None, *,
                     dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
                     tile: int = 0):
    """y [m, n] = x . w^T (+ bias) in `dtype` over two quantized tensors. `tile`
    != 0 forces a kernel variant (test / tuning hook)."""
    dt = _dtype16(dtype)
    m, k, xc, xs, dev = _quantized(x_codes, x_scales, "x_")
    n, kw, wc, ws, dev_w = _quantized(w_codes, w_scales, "w_")
    if kw != k or dev_w != dev:
        raise ValueError(f"x_codes [{m}, {k // 2}] on device {dev} do not fit w_codes "
                         f"[{n}, {kw // 2}] on device {dev_w}")
    pb = None if bias is None else _tensor(bias, "bias", dtype, (n,), dev)
    out, po = _output(out, "out", (m, n), dtype, x_codes)
    _launch("convrot_gemm_mx4", dev, xc, xs, wc, ws, pb, m, n, k, po, dt, tile)
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
    n, kw, wc, ws, dev = _quantized(w_codes, w_scales, "w_")
    if kw != k or x.get_device() != dev:
        raise ValueError(f"x [{m}, {k}] on {x.device} does not fit w_codes [{n}, {kw // 2}] on "
                         f"{w_codes.device}")
    pb = None if bias is None else _tensor(bias, "bias", x.dtype, (n,), dev)
    if workspace is None:
        size = load_library().convrot_linear_mx4_workspace_size(m, n, k)
        workspace = torch.empty_strided((size,), (1,), dtype=_U8, device=x.device)
        pw = workspace.data_ptr()
    else:
        pw = _tensor(workspace, "workspace", _U8, (workspace.numel(),), dev)
        size = workspace.numel()
    out, po = _output(out, "out", (m, n), x.dtype, x)
    _launch("convrot_linear_mx4", dev, x.data_ptr(), wc, ws, pb, m, n, k, g, rot_seed, po, dt, pw,
            size)
    return out


def _modulation(t, name: str, x: torch.Tensor, m: int, k: int, samples: int):
    """Check a modulation ([k] or [b, k], rows of any stride) against the `samples`
    of those before it (0: none yet); (address, row stride, samples)."""
    if not isinstance(t, torch.Tensor) or t.dtype != x.dtype:
        raise TypeError(f"{name} must be a {x.dtype} tensor")
    shape, strides = t.shape, t.stride()
    if t.get_device() != x.get_device():
        raise ValueError(f"{name} is on {t.device}, expected {x.device}")
    if len(shape) not in (1, 2) or shape[-1] != k or strides[-1] != 1:
        raise ValueError(f"{name} must be [{k}] or [samples, {k}] with contiguous rows "
                         f"(got shape {tuple(shape)}, strides {strides})")
    b = shape[0]
    if len(shape) == 1 or b == 1:
        return t.data_ptr(), 0, samples
    if samples not in (0, b):
        raise ValueError(f"{name} has {b} samples, another modulation {samples}")
    if b == 0 or m % b:
        raise ValueError(f"{m} rows do not divide into {b} samples")
    return t.data_ptr(), strides[0], b


def _norm_args(x, o, gate, post_norm, post_weight, norm, weight, scale, shift, eps, x_out):
    dt = _input16(x, "x")
    m, k = x.shape
    dev, dtype = x.get_device(), x.dtype
    if norm not in ("rms", "layer") or post_norm not in _NORMS:
        raise ValueError(f"norm={norm!r}, post_norm={post_norm!r}: 'rms' or 'layer'")
    a = _NormArgs(x=x.data_ptr(), m=m, k=k, dtype=dt, norm=_NORMS[norm],
                  post_norm=_NORMS[post_norm], eps=eps)
    if o is not None:
        a.o = _tensor(o, "o", dtype, (m, k), dev)
        x_out, a.x_out = _output(x_out, "x_out", (m, k), dtype, x)
    elif x_out is not None or gate is not None or post_norm is not None:
        raise ValueError("x_out, gate and post_norm need o")
    else:
        x_out = x
    if post_weight is not None:
        a.post_weight = _tensor(post_weight, "post_weight", dtype, (k,), dev)
    if weight is not None:
        a.weight = _tensor(weight, "weight", dtype, (k,), dev)
    samples = 0
    if gate is not None:
        a.gate, a.gate_stride, samples = _modulation(gate, "gate", x, m, k, samples)
    if scale is not None:
        a.scale, a.scale_stride, samples = _modulation(scale, "scale", x, m, k, samples)
    if shift is not None:
        a.shift, a.shift_stride, samples = _modulation(shift, "shift", x, m, k, samples)
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
    h, a.h = _output(h, "h", x.shape, x.dtype, x)
    _launch("convrot_norm_residual", x.get_device(), ctypes.byref(a))
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
    codes, scales, a.h_codes, a.h_scales = _new_quantized(*x.shape, x, codes, scales)
    a.g, a.rot_seed = g, rot_seed
    if h is not None:
        a.h = _tensor(h, "h", x.dtype, x.shape, x.get_device())
    _launch("convrot_norm_residual", x.get_device(), ctypes.byref(a))
    return x_out, codes, scales
