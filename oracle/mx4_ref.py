"""CPU oracle of the microscaled 4-bit (MXFP4) layers and the gated residual
norm: numpy in float64, sharing no code with the library.

Inputs are float64 arrays holding bf16 or half values. The rotation is a dense
matrix product with R = H_g . diag(d) / sqrt(g), exact in float64 for inputs
whose nonzero magnitudes span at most 37 binades within a group (products by
+-1, at most 256 terms of 8 bits; half inputs always); a caller that feeds wider
groups gets the float64 sum, like the library's contract.
"""

from __future__ import annotations

import numpy as np

from .convrot_ref import hadamard, rotation_signs

# magnitudes by code, and the midpoints between neighbours (ties go to the even code)
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = 32


def rotation(g: int, seed: int) -> np.ndarray:
    """R [g, g]; g = 1: the identity."""
    if g == 1:
        return np.ones((1, 1))
    return hadamard(g).astype(np.float64) * np.asarray(rotation_signs(seed, g), np.float64) \
        / np.sqrt(g)


def rotate(x: np.ndarray, g: int, seed: int) -> np.ndarray:
    """x . blockdiag(R), each element's sum rounded once to fp32."""
    rows, k = x.shape
    with np.errstate(invalid="ignore", over="ignore"):
        y = x.reshape(rows, k // g, g) @ rotation(g, seed) if g > 1 else x
        return y.reshape(rows, k).astype(np.float32)


def encode(v: np.ndarray):
    """fp32 [rows, k] -> (codes 0..15 uint8 [rows, k], exponent bytes uint8
    [rows, k/32]), the sign bit set for negative values that do not round to 0."""
    rows, k = v.shape
    b = v.astype(np.float64).reshape(rows, k // BLOCK, BLOCK)
    with np.errstate(invalid="ignore", divide="ignore"):
        top = np.abs(b).max(-1)          # NaN stays NaN
        bad = ~np.isfinite(top)
        # floor(log2) from the exact binary representation
        e = np.frexp(np.where(bad | (top == 0), 1.0, top))[1] - 1 - 2
        e = np.maximum(np.where(top == 0, -127, e), -127)
        u = np.ldexp(np.where(bad[..., None], 0.0, b), -e[..., None])
    a = np.abs(u)
    # nearest magnitude; between two equally near ones the even code
    d = np.abs(a[..., None] - MAGNITUDES)
    order = np.argsort(np.where(np.arange(8) % 2 == 0, 0, 1), kind="stable")  # even codes first
    code = order[np.argmin(d[..., order], -1)].astype(np.uint8)
    code = np.where(a >= 6.0, 7, code).astype(np.uint8)
    code |= np.where((u < 0) & (code > 0), 8, 0).astype(np.uint8)
    return code.reshape(rows, k), np.where(bad, 255, e + 127).astype(np.uint8)


def values(code: np.ndarray, exps: np.ndarray) -> np.ndarray:
    """float64 [rows, k] that codes and exponent bytes stand for."""
    mag = np.where(code & 8, -1.0, 1.0) * MAGNITUDES[code & 7]
    unit = np.where(exps == 255, np.nan, np.ldexp(1.0, exps.astype(np.int64) - 127))
    return mag * np.repeat(unit, BLOCK, -1)


def pack(code: np.ndarray, exps: np.ndarray, fill: int = 0):
    """The held form: codes [rows, k/2], scales [ceil(k/256), rows16, 8]."""
    rows, k = code.shape
    codes = (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8)
    rows16, tiles = -(-rows // 16) * 16, -(-k // 256)
    scales = np.full((tiles, rows16, 8), fill, np.uint8)
    for b in range(k // BLOCK):
        scales[b // 8, :rows, b % 8] = exps[:, b]
    return codes, scales


def unpack(codes: np.ndarray, scales: np.ndarray):
    """Inverse of pack."""
    rows, half = codes.shape
    code = np.empty((rows, 2 * half), np.uint8)
    code[:, 0::2] = codes & 15
    code[:, 1::2] = codes >> 4
    nb = 2 * half // BLOCK
    exps = np.stack([scales[b // 8, :rows, b % 8] for b in range(nb)], 1)
    return code, exps


def quantize(x: np.ndarray, g: int, seed: int):
    return encode(rotate(x, g, seed))


def derotate(v: np.ndarray, g: int, seed: int) -> np.ndarray:
    """v . blockdiag(R)^T in float64."""
    rows, k = v.shape
    if g == 1:
        return v
    return (v.reshape(rows, k // g, g) @ rotation(g, seed).T).reshape(rows, k)


def norm(v: np.ndarray, kind: str, weight=None, eps: float = 1e-6) -> np.ndarray:
    if kind == "layer":
        v = v - v.mean(-1, keepdims=True)
    v = v / np.sqrt((v * v).mean(-1, keepdims=True) + eps)
    return v if weight is None else v * weight


def per_row(mod: np.ndarray, m: int) -> np.ndarray:
    """A modulation row per sample -> one per row of x."""
    mod = np.atleast_2d(mod)
    return np.repeat(mod, m // mod.shape[0], 0)
