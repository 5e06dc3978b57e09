"""The MXFP4 and norm entry points without a GPU: refusals come before any HIP
call, sizes and launch plans are host arithmetic, and the oracle's own pins."""

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import int8_gemm_amd as cr
from int8_gemm_amd import mx4
from oracle import mx4_ref as ref


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(cr.library_path()):
        from int8_gemm_amd import _build
        _build.build()
    return cr.load_library()


# aligned stand-ins, far apart, never dereferenced on these paths
A, B, C, D, E, F = (1 << 32, 1 << 36, 1 << 40, 1 << 42, 1 << 44, 1 << 46)


@pytest.mark.parametrize("g,k,want", [(512, 512, 2), (0, 256, 2), (2, 256, 2), (64, 96, 2),
                                      (256, 320, 2), (1, 16, 3), (4, 100, 3), (1, 131104, 3),
                                      (1, 0, 1), (1, -32, 1)])
def test_bad_groups_and_shapes(lib, g, k, want):
    assert lib.convrot_quantize_mx4(A, 0, 8, k, g, 1, B, C, None) == want
    assert lib.convrot_dequant_mx4(A, B, 8, k, g, 1, C, 0, None) == want
    assert lib.convrot_linear_mx4(A, B, C, None, 8, 16, k, g, 1, D, 0, E, 1 << 30, None) == want
    assert lib.convrot_last_error_string()


def test_quantize_and_dequant_refusals(lib):
    q, d = lib.convrot_quantize_mx4, lib.convrot_dequant_mx4
    assert q(A, 2, 8, 256, 1, 1, B, C, None) == 1          # format
    assert q(A, 0, -1, 256, 1, 1, B, C, None) == 1
    assert q(A, 0, 1 << 31, 256, 1, 1, B, C, None) == 3
    # grids count their threads in 32 bits
    assert q(A, 0, 1 << 29, 32, 1, 1, B, C, None) == 3
    assert d(A, B, 1 << 20, 131072, 1, 1, C, 0, None) == 3
    for bad in ((None, B, C), (A, None, C), (A, B, None)):
        assert q(bad[0], 0, 8, 256, 1, 1, bad[1], bad[2], None) == 1
        assert d(bad[0], bad[1], 8, 256, 1, 1, bad[2], 0, None) == 1
    for bad in ((A + 8, B, C), (A, B + 8, C), (A, B, C + 8)):
        assert q(bad[0], 0, 8, 256, 1, 1, bad[1], bad[2], None) == 4
        assert d(bad[0], bad[1], 8, 256, 1, 1, bad[2], 0, None) == 4
    assert q(A, 0, 8, 256, 1, 1, A + 4080, C, None) == 1    # codes in x
    assert q(A, 0, 8, 256, 1, 1, B, B + 1008, None) == 1    # scales in codes
    assert d(A, B, 8, 256, 1, 1, A + 1008, 0, None) == 1    # out in codes
    assert d(A, B, 8, 256, 1, 1, B + 112, 0, None) == 1     # out in scales (16 rows held)
    assert q(None, 0, 0, 256, 1, 1, None, None, None) == 0  # no rows
    assert d(None, None, 0, 256, 1, 1, None, 0, None) == 0


def test_gemm_refusals(lib):
    def gemm(xc=A, xs=B, wc=C, ws=D, bias=None, m=8, n=32, k=256, y=E, dt=0, tile=0):
        return lib.convrot_gemm_mx4(xc, xs, wc, ws, bias, m, n, k, y, dt, tile, None)
    assert gemm(dt=7) == 1
    for tile in (-1, 1, 8, 32, 48, 100, 512):
        assert gemm(tile=tile) == 1
    assert gemm(m=65, tile=16) == 1   # more rows than it holds
    assert gemm(n=24) == 3 and gemm(k=272) == 3 and gemm(k=131104) == 3
    assert gemm(n=0) == 1 and gemm(k=0) == 1 and gemm(m=-1) == 1
    assert gemm(m=1 << 30, n=1 << 30) == 3 and gemm(m=(1 << 31) - 1) == 3
    assert gemm(n=1 << 27) == 3 and gemm(m=1 << 30, n=16, k=32) == 3
    for name in ("xc", "xs", "wc", "ws", "y"):
        assert gemm(**{name: None}) == 1
        assert gemm(**{name: F + 8}) == 4
    assert gemm(bias=F + 4) == 4
    for inside in ({"xc": E + 496}, {"xs": E + 496}, {"wc": E + 496}, {"ws": E + 496},
                   {"bias": E + 504}):
        assert gemm(**inside) == 1                          # y is 8 x 32 16-bit values
    assert gemm(m=0, xc=None, xs=None, y=None) == 0
    assert gemm(m=0, wc=None) == 1


def test_linear_refusals_and_workspace(lib):
    size = cr.convrot_linear_mx4_workspace_for_rows
    assert size(1, 256) == 256 + 16 * 8 and size(3, 320) == 512 + 2 * 16 * 8
    assert size(17, 256) == 17 * 128 + 128 + 32 * 8          # codes rounded up to 256
    assert size(0, 256) == 0 and size(1, 0) == 0
    rows = (64 << 20) // (128 + 8)      # at least 64 MiB ...
    assert cr.convrot_linear_mx4_workspace_size(10 ** 6, 16, 256) == size(rows, 256)
    # ... or three rows per output column
    assert cr.convrot_linear_mx4_workspace_size(10 ** 6, 1 << 18, 256) == size(3 << 18, 256)
    assert cr.convrot_linear_mx4_workspace_size(10, 16, 256) == size(10, 256)
    assert cr.convrot_linear_mx4_workspace_size(0, 16, 256) == size(1, 256)
    assert cr.convrot_mx4_scales_size(17, 288) == 2 * 32 * 8

    def lin(x=A, wc=B, ws=C, bias=None, m=8, n=32, k=256, g=256, y=D, dt=0, w=E, size=1 << 20):
        return lib.convrot_linear_mx4(x, wc, ws, bias, m, n, k, g, 1, y, dt, w, size, None)
    assert lin(size=256 + 127) == 5                          # one row needs 384
    assert lin(w=E + 128) == 4 and lin(x=A + 2) == 4 and lin(y=D + 2) == 4
    assert lin(x=None) == 1 and lin(wc=None) == 1 and lin(y=None) == 1 and lin(w=None) == 1
    assert lin(y=A + 16) == 1 and lin(x=E + 512) == 1 and lin(wc=E + 512) == 1
    assert lin(bias=E + 512) == 1 and lin(y=E + 512) == 1 and lin(bias=D + 8) == 1
    assert lin(dt=3) == 1 and lin(n=40) == 3 and lin(g=512) == 2
    assert lin(m=0, x=None, y=None, w=None, size=0) == 0


def norm_status(lib, **kw):
    a = mx4._NormArgs(x=A, o=B, x_out=C, h=D, m=8, k=256, rows_per_mod=8, norm=1, eps=1e-6)
    for name, v in kw.items():
        setattr(a, name, v)
    return lib.convrot_norm_residual(ctypes.byref(a), None)


def test_norm_refusals(lib):
    def st(**kw):
        return norm_status(lib, **kw)
    assert lib.convrot_norm_residual(None, None) == 1
    assert st(dtype=2) == 1 and st(norm=0) == 1 and st(norm=3) == 1 and st(post_norm=4) == 1
    assert st(eps=float("nan")) == 1 and st(eps=-1.0) == 1 and st(eps=float("inf")) == 1
    assert st(m=-1) == 1 and st(k=0) == 1 and st(k=12) == 3 and st(k=16392) == 3
    assert st(m=1 << 31) == 3 and st(m=1 << 26, k=8) == 3 and st(m=1 << 25, k=2056) == 3
    assert st(x=None) == 1 and st(h=None) == 1 and st(x_out=None) == 1
    # what needs o
    assert st(o=None) == 1 and st(o=None, x_out=None, gate=E) == 1
    assert st(o=None, x_out=None, post_norm=1) == 1 and st(post_weight=E) == 1
    # quantized h: both buffers, a group that divides k
    assert st(h_codes=E, g=1) == 1 and st(h_scales=E, g=1) == 1
    assert st(h_codes=E, h_scales=F, g=0) == 2 and st(h_codes=E, h_scales=F, g=256, k=320) == 2
    assert st(h_codes=E, h_scales=F, g=1, k=40) == 3
    # alignment and strides
    for name in ("x", "o", "x_out", "weight", "gate", "scale", "shift", "h"):
        assert st(**{name: F + 8}) == 4, name
    assert st(gate=E, gate_stride=4) == 4 and st(gate=E, gate_stride=-8) == 1
    assert st(gate=E, rows_per_mod=0) == 1
    # overlaps: outputs with inputs and with each other (8 rows of 512 bytes)
    for kw in ({"x_out": A + 512}, {"x_out": B}, {"h": A}, {"h": B + 16}, {"h": C + 4080},
               {"weight": C + 16}, {"post_weight": D, "post_norm": 1}, {"gate": D + 4080},
               {"scale": C - 256}, {"shift": C - 4096, "rows_per_mod": 1, "shift_stride": 512},
               {"h_codes": C, "h_scales": F, "g": 1}, {"h_codes": E, "h_scales": E + 16, "g": 1}):
        assert st(**kw) == 1, kw
    assert st(m=0, x=None, o=None, x_out=None, h=None) == 0


def test_binding_checks_tensors():
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    u8 = torch.zeros((4, 128), dtype=torch.uint8)
    sc = torch.zeros((1, 16, 8), dtype=torch.uint8)
    with pytest.raises(ValueError):          # no device tensors
        cr.convrot_quantize_mx4(x, 256)
    with pytest.raises(ValueError):
        cr.convrot_dequant_mx4(u8, sc, 256)
    with pytest.raises(ValueError):
        cr.convrot_gemm_mx4(u8, sc, u8, sc)
    with pytest.raises(ValueError):
        cr.convrot_norm_residual(x)
    with pytest.raises(TypeError):
        cr.convrot_quantize_mx4(x.float(), 256)
    with pytest.raises(TypeError):
        cr.convrot_dequant_mx4(u8, sc, 256, dtype=torch.float32)
    with pytest.raises(ValueError):
        mx4._tensor(x, "x", torch.bfloat16, (4, 128), -1)
    with pytest.raises(ValueError):
        mx4._tensor(x.t(), "x", torch.bfloat16, (256, 4), -1)


def test_binding_checks_modulations():
    x = torch.zeros((8, 64), dtype=torch.bfloat16)
    mod = torch.zeros((4, 192), dtype=torch.bfloat16)

    def call(t, samples=0):
        return mx4._modulation(t, "gate", x, 8, 64, samples)
    assert call(mod[:, 64:128]) == (mod.data_ptr() + 128, 192, 4)
    assert call(mod[:1, :64]) == (mod.data_ptr(), 0, 0) and call(mod[0, :64], 4)[1:] == (0, 4)
    with pytest.raises(TypeError):
        call(mod.float())
    for bad, samples in ((mod, 0), (mod[:3, :64], 0), (mod[:, :64], 2), (mod[:, ::3], 0),
                         (mod[:0, :64], 0), (mod[None, :, :64], 0)):
        with pytest.raises(ValueError):
            call(bad, samples)


@pytest.mark.parametrize("cus", [256, 128, 3])
def test_gemm_plans(lib, cus):
    """Up to 64 rows take the few-rows kernel (blocks of 16 to 64 columns) or
    tiles, by the shape alone; more rows take tiles."""
    for m, n, k, few in ((1, 3840, 3840, True), (16, 5120, 13824, True), (64, 16, 256, True),
                         (64, 13824, 5120, False), (32, 11520, 3840, False), (40, 512, 8192, True)):
        p = cr.convrot_plan_launch("gemm_mx4", m=m, n=n, k=k, compute_units=cus)
        assert (p["tile_m"] == 16) == few
        if few:
            assert p["tile_n"] in (16, 32, 64) and p["grid"] == -(-n // p["tile_n"])
    for m in (65, 1000, 32760):
        p = cr.convrot_plan_launch("gemm_mx4", m=m, n=3840, k=3840, compute_units=cus)
        assert p["tile_m"] in (64, 128, 192, 256, 384)
        assert p["grid"] == -(-m // p["tile_m"]) * -(-3840 // p["tile_n"])
    with pytest.raises(cr.ConvrotError, match="UNSUPPORTED_SHAPE"):
        cr.convrot_plan_launch("gemm_mx4", m=8, n=24, k=64, compute_units=cus)


def test_header_compiles_and_links_as_c99(lib, tmp_path):
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("no gcc")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = os.path.join(root, "tests", "c", "header_mx4_c99.c")
    r = subprocess.run([cc, "-std=c99", "-pedantic", "-Wall", "-Werror", "-fPIC", "-shared",
                        "-I", os.path.join(root, "include"), src, "-o", str(tmp_path / "h.so"),
                        cr.library_path(), "-Wl,--no-undefined",
                        "-Wl,--unresolved-symbols=ignore-in-shared-libs"],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_norm_args_match_the_header(lib, tmp_path):
    """The binding's structure has the size and offsets of convrot_norm_args."""
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("no gcc")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    fields = [f for f, _ in mx4._NormArgs._fields_]
    src = tmp_path / "o.c"
    src.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"convrot.h\"\nint main(void) {"
                   + "".join(f'printf("%zu ", offsetof(convrot_norm_args, {f}));' for f in fields)
                   + 'printf("%zu", sizeof(convrot_norm_args)); return 0; }')
    exe = tmp_path / "o"
    subprocess.run([cc, "-std=c99", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)],
                   check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    assert got == [getattr(mx4._NormArgs, f).offset for f in fields] \
        + [ctypes.sizeof(mx4._NormArgs)]


def test_oracle_pins():
    v = np.array([[0, .25, .26, .75, 1.25, 1.26, 1.75, 2.5, 2.51, 3.5, 5, 5.01, 6, 7.9, -5, -.25]
                  * 2], np.float32)
    c, e = ref.encode(v)
    assert e.tolist() == [[127]]
    assert ref.values(c, e)[0, :16].tolist() == [0, 0, .5, 1, 1, 1.5, 2, 2, 3, 4, 4, 6, 6, 6, -4, 0]
    # powers of two, the clamp at 2^-127, zeros
    for top, want in ((8.0, 128), (7.99, 127), (2.0 ** -125, 0), (2.0 ** -149, 0), (0.0, 0)):
        x = np.zeros((1, 32), np.float32)
        x[0, 3] = top
        assert ref.encode(x)[1][0, 0] == want
    for g in (4, 16, 64, 256):
        r = ref.rotation(g, 0xC0FFEE)
        assert np.array_equal(r @ r.T, np.eye(g))
    rng = np.random.default_rng(0)
    code = rng.integers(0, 16, (5, 288)).astype(np.uint8)
    exps = rng.integers(0, 255, (5, 9)).astype(np.uint8)
    codes, scales = ref.pack(code, exps)
    assert codes.shape == (5, 144) and scales.shape == (2, 16, 8)
    back = ref.unpack(codes, scales)
    assert np.array_equal(back[0], code) and np.array_equal(back[1], exps)


def test_gemm_grids_of_many_tiles(lib):
    """Grids count their threads in 32 bits: a forced small tile is refused where
    there are too many, and the automatic choice passes it over."""
    def gemm(m, n, tile):
        return lib.convrot_gemm_mx4(A, B, C, D, None, m, n, 32, E, 0, tile, None)
    m, n = 64 << 13, 64 << 10       # 2^23 tiles of 64 x 64
    assert gemm(m, n, 64) == 3 and gemm(m, n, 40) == 3
    assert gemm(2 * m, n, 0) == 3   # 2^24: beyond the documented sizes
    for cus in (256, 1):
        p = cr.convrot_plan_launch("gemm_mx4", m=2 * m - 64, n=n, k=32, compute_units=cus)
        assert p["grid"] * p["block"] < 1 << 32
        assert p["tile_m"] * p["tile_n"] > 64 * 64


def test_norm_modulation_ranges_do_not_overflow(lib):
    """rows_per_mod beyond m means one row for all, whose range is one row long; a
    range that 64 bits do not hold is refused."""
    def st(**kw):
        return norm_status(lib, **kw)
    for rows in (8, 9, 1 << 40, (1 << 63) - 1):
        # D: the 8 rows of h; the modulation lies in its first row, or its last
        assert st(gate=D + 16, gate_stride=512, rows_per_mod=rows) == 1, rows
        assert st(scale=D + 4080, scale_stride=512, rows_per_mod=rows) == 1, rows
    big = {"m": (1 << 25) - 8, "x": 1 << 52, "o": 1 << 53, "x_out": 1 << 54, "h": 1 << 50}
    assert st(shift=(1 << 50) + 16, shift_stride=1 << 40, rows_per_mod=1, **big) == 1
    assert st(shift=E, shift_stride=1 << 60, rows_per_mod=1) == 1


def test_sizes_of_invalid_dimensions_are_zero(lib):
    rows, size = cr.convrot_linear_mx4_workspace_for_rows, cr.convrot_linear_mx4_workspace_size
    far = 1 << 31
    for k in (0, -32, 16, 100, 131104):
        assert rows(8, k) == 0 and size(8, 16, k) == 0 and cr.convrot_mx4_scales_size(8, k) == 0, k
    for m in (-1, far, 1 << 62):
        assert rows(m, 256) == 0 and size(m, 16, 256) == 0
        assert cr.convrot_mx4_scales_size(m, 256) == 0
    for n in (0, -16, 24, far, (1 << 62) + 16, (1 << 63) - 16):
        assert size(8, n, 256) == 0, n
    assert size(8, 16, 131072) == rows(8, 131072) > 0


@pytest.mark.parametrize("rows,k", [(16, 256), (5, 2880), (33, 288), (48, 512)])
def test_row_major_scales_are_brought_into_the_held_order(rows, k):
    """The header's recipe: pad to multiples of 16 rows and 8 columns, with any bytes,
    reshape, swap the first two axes."""
    rng = np.random.default_rng(rows)
    exps = rng.integers(0, 256, (rows, k // 32)).astype(np.uint8)
    padded = np.pad(exps, ((0, -rows % 16), (0, -(k // 32) % 8)), constant_values=7)
    held = padded.reshape(padded.shape[0], -1, 8).swapaxes(0, 1)
    codes, want = ref.pack(np.zeros((rows, k), np.uint8), exps)
    assert held.shape == want.shape == mx4._scales_shape(rows, k)
    assert np.array_equal(ref.unpack(codes, held)[1], exps)
    assert held.size == cr.convrot_mx4_scales_size(rows, k)
