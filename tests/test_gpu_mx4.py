"""GPU: the microscaled 4-bit (MXFP4) layers against a float64 oracle.

Quantization is compared exactly. For the others the bounds count roundings
(u = 2^-24 an fp32 half step; h16 the half step of the output format relative
to the value, plus half of its smallest subnormal):
  dequant   log2(g) additions per output in fp32, each off by at most u times a
            partial sum of |v|, then one rounding to 16 bits;
  gemm      k exact products summed in fp32 in some order: at most k u sum|x w|,
            one more addition for the bias, then one rounding to 16 bits.
"""

import numpy as np
import pytest
import torch

import int8_gemm_amd as cr
import synth
from oracle import mx4_ref as ref

pytestmark = pytest.mark.gpu

SEED = synth.ROT_SEED
DEV = "cuda:0"
U = 2.0 ** -24
H16 = {torch.bfloat16: (2.0 ** -8, 2.0 ** -134), torch.float16: (2.0 ** -11, 2.0 ** -25)}
MAX16 = {torch.bfloat16: float(torch.finfo(torch.bfloat16).max), torch.float16: 65504.0}
DTYPES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    cr.load_library()


def dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).to(DEV)


def f64(t):
    return t.cpu().to(torch.float64).numpy()


def tokens(rng, m, k, outliers=True):
    x = rng.standard_normal((m, k))
    if outliers:
        x[:, rng.integers(0, k, max(1, k // 100))] *= 30
    return x


def held(rng, rows, k, lo=118, hi=134, fill=0):
    """A random quantized tensor: codes and scales as held, and its values."""
    code = rng.integers(0, 16, (rows, k)).astype(np.uint8)
    exps = rng.integers(lo, hi, (rows, k // 32)).astype(np.uint8)
    c, s = ref.pack(code, exps, fill)
    return torch.from_numpy(c).to(DEV), torch.from_numpy(s).to(DEV), ref.values(code, exps)


def assert_quantized(codes, scales, x64, g, seed=SEED):
    want_c, want_e = ref.quantize(x64, g, seed)
    got_c, got_e = ref.unpack(codes.cpu().numpy(), scales.cpu().numpy())
    assert np.array_equal(got_e, want_e)
    a, b = ref.values(got_c, got_e), ref.values(want_c, want_e)
    assert np.array_equal(a[~np.isnan(b)], b[~np.isnan(b)])
    assert np.array_equal(np.isnan(a), np.isnan(b))


# ---- quantize ---------------------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f16"])
@pytest.mark.parametrize("g,m,k", [
    (1, 1, 32), (1, 3, 96), (1, 33, 288), (4, 1, 32), (4, 17, 224), (16, 9, 480), (16, 130, 512),
    (64, 1, 64), (64, 31, 320), (64, 8, 5120), (256, 1, 256), (256, 1, 5120), (256, 7, 768),
    (256, 100, 3840), (256, 40, 13824)])
def test_quantize_matches_oracle(g, m, k, dtype):
    rng = np.random.default_rng(g * 1000 + m + k)
    x = dev(tokens(rng, m, k), dtype)
    codes, scales = cr.convrot_quantize_mx4(x, g, SEED)
    assert_quantized(codes, scales, f64(x), g)


@pytest.mark.parametrize("g", [1, 4, 16, 64, 256])
def test_quantize_wide_spans_ties_and_zero_blocks(g):
    """Magnitudes over 36 binades of a group (28 and the 8 bits of each), exact ties, powers of two, rows of
    zeros, and a row with a single nonzero element."""
    rng = np.random.default_rng(g)
    k = 1024
    x = rng.uniform(1, 2, (24, k)) * rng.choice([-1, 1], (24, k))
    x *= np.exp2(rng.integers(-14, 15, (24, k)))
    x[1] = 0
    x[2] = 0
    x[2, 700] = -3.0
    x[3] = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, -0.25, -5.0], k)
    x[4] = np.exp2(rng.integers(-3, 3, k)) * rng.choice([-1, 1], k)
    x[5, :] = 1.0
    x[6] = np.tile([1.0, -1.0], k // 2)
    x[7] = rng.integers(-3, 4, k)
    x[8] = 0
    x[8, ::256] = rng.integers(-40, 40, 4)
    t = dev(x, torch.bfloat16)
    codes, scales = cr.convrot_quantize_mx4(t, g, SEED)
    assert_quantized(codes, scales, f64(t), g)


@pytest.mark.parametrize("exp", [-133, -128, -126, -125, -120, 100, 120, 123])
@pytest.mark.parametrize("g", [1, 16, 256])
def test_quantize_at_the_ends_of_the_range(g, exp):
    rng = np.random.default_rng(exp + 200)
    x = dev(rng.integers(-7, 8, (16, 512)) * np.exp2(float(exp)), torch.bfloat16)
    codes, scales = cr.convrot_quantize_mx4(x, g, SEED)
    assert_quantized(codes, scales, f64(x), g)


@pytest.mark.parametrize("exp", [-24, -22, -17, -14, 8, 12])
@pytest.mark.parametrize("g", [1, 4, 16, 256])
def test_quantize_half_at_the_ends_of_its_range(g, exp):
    """Subnormal halves among them; every half value and sign."""
    rng = np.random.default_rng(exp + 300)
    x = dev(rng.integers(-15, 16, (16, 512)) * 2.0 ** exp, torch.float16)
    codes, scales = cr.convrot_quantize_mx4(x, g, SEED)
    assert_quantized(codes, scales, f64(x), g)
    every = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.float16)
    every = every[torch.isfinite(every)].reshape(-1, 2048).to(DEV)
    assert_quantized(*cr.convrot_quantize_mx4(every, g, SEED), f64(every), g)


@pytest.mark.parametrize("g", [1, 64, 256])
def test_quantize_marks_blocks_that_are_not_finite(g):
    rng = np.random.default_rng(5)
    x = rng.standard_normal((9, 768))
    x[1, 3] = np.nan
    x[2, 300] = np.inf
    x[3, 767] = -np.inf
    x[4, 10], x[4, 11] = np.inf, -np.inf
    t = dev(x, torch.bfloat16)
    codes, scales = cr.convrot_quantize_mx4(t, g, SEED)
    assert_quantized(codes, scales, f64(t), g)
    # ... and they come back as NaN, through the product too
    w = cr.convrot_quantize_mx4(dev(rng.standard_normal((16, 768)), torch.bfloat16), g, SEED)
    y = cr.convrot_gemm_mx4(codes, scales, *w)
    assert torch.isnan(y).all(-1).cpu().tolist() == [False, True, True, True, True] + [False] * 4
    big = torch.cat([codes] * 8)
    sc = torch.zeros((3, 80, 8), dtype=torch.uint8, device=DEV)
    for r in range(8):
        sc[:, 9 * r:9 * r + 9] = scales[:, :9]
    y = cr.convrot_gemm_mx4(big, sc, *w)    # the tiled kernel
    assert torch.isnan(y).all(-1).cpu().tolist() == \
        ([False, True, True, True, True] + [False] * 4) * 8


def test_quantize_leaves_padding_rows_and_what_lies_behind():
    rng = np.random.default_rng(6)
    m, k = 5, 96
    x = dev(rng.standard_normal((m, k)), torch.bfloat16)
    codes = torch.full((m + 3, k // 2), 77, dtype=torch.uint8, device=DEV)
    scales = torch.full((1, 16, 8), 77, dtype=torch.uint8, device=DEV)
    cr.convrot_quantize_mx4(x, 16, SEED, codes=codes[:m], scales=scales)
    assert (codes[m:] == 77).all() and (scales[:, m:] == 77).all()
    assert (scales[:, :m, 3:] == 0).all()
    assert_quantized(codes[:m], scales, f64(x), 16)


@pytest.mark.parametrize("g", [4, 16, 64, 256])
def test_quantize_of_values_on_every_border(g):
    """Small integers and repeated values: most rotated elements lie on borders
    of codes or exponents, where sums in fp32 with an error bound decide nothing."""
    rng = np.random.default_rng(g)
    k = 2048
    x = np.zeros((40, k))
    x[:8] = rng.integers(-2, 3, (8, k))
    x[8:12] = rng.choice([-1.0, 1.0], (4, k))
    x[12:16] = np.repeat(rng.integers(-9, 10, (4, k // 64)), 64, -1)
    x[16:20, ::g] = rng.integers(-9, 10, (4, k // g))
    x[20] = 1.0
    x[21] = 2.0 ** -60
    x[22:30] = rng.integers(-128, 129, (8, k)) * 2.0 ** 40
    x[30:, :1024] = rng.standard_normal((10, 1024))    # half a row of zeros
    for dtype in DTYPES:
        t = dev(np.where(np.abs(x) < 60000, x, 1.0) if dtype == torch.float16 else x, dtype)
        codes, scales = cr.convrot_quantize_mx4(t, g, SEED)
        assert_quantized(codes, scales, f64(t), g)


@pytest.mark.parametrize("seed", [0, 2 ** 64 - 1])
def test_quantize_takes_the_rotation_seed(seed):
    rng = np.random.default_rng(7)
    x = dev(tokens(rng, 10, 512), torch.bfloat16)
    assert_quantized(*cr.convrot_quantize_mx4(x, 64, seed), f64(x), 64, seed)


# ---- dequant ----------------------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f16"])
@pytest.mark.parametrize("g,rows,k", [(1, 1, 32), (1, 35, 352), (4, 5, 96), (16, 16, 288),
                                      (64, 33, 576), (256, 1, 256), (256, 70, 3840)])
def test_dequant_matches_oracle(g, rows, k, dtype):
    rng = np.random.default_rng(rows + k)
    codes, scales, v = held(rng, rows, k, fill=255)   # padding bytes are never used
    out = f64(cr.convrot_dequant_mx4(codes, scales, g, SEED, dtype=dtype))
    want = ref.derotate(v, g, SEED)
    # |terms| of an output: its group's |v| / sqrt(g)
    mass = np.repeat(np.abs(v).reshape(rows, k // g, g).sum(-1), g, -1) / np.sqrt(g)
    half, tiny = H16[dtype]
    tol = half * np.abs(want) + tiny + (np.log2(g) * U * mass if g > 1 else 0)
    assert (np.abs(out - want) <= tol).all()


def test_dequant_of_the_whole_exponent_range():
    """Every exponent byte against every code: exact where the format holds it."""
    code = np.tile(np.arange(16, dtype=np.uint8), (256, 2))
    exps = np.arange(256, dtype=np.uint8)[:, None]
    c, s = ref.pack(code, exps)
    out = cr.convrot_dequant_mx4(torch.from_numpy(c).to(DEV), torch.from_numpy(s).to(DEV), 1)
    want = torch.from_numpy(ref.values(code, exps)).to(torch.float32).to(torch.bfloat16)
    assert torch.equal(torch.nan_to_num(out.cpu().float(), nan=7.0),
                       torch.nan_to_num(want.float(), nan=7.0))
    assert torch.isnan(out[255]).all() and not torch.isnan(out[:255]).any()


@pytest.mark.parametrize("g", [4, 16, 64, 256])
def test_read_back_is_near_the_input(g):
    """Round trip: 4 bits hold a value to 1/4 of its own size or 1/4 unit; over a
    group the rotation is orthogonal, so the 2-norm error carries over."""
    rng = np.random.default_rng(g)
    x = dev(tokens(rng, 64, 2048), torch.bfloat16)
    back = f64(cr.convrot_dequant_mx4(*cr.convrot_quantize_mx4(x, g, SEED), g, SEED))
    c, e = ref.quantize(f64(x), g, SEED)
    want = ref.derotate(ref.values(c, e), g, SEED)
    # half a step of bf16, and fp32 sums far below it
    assert np.linalg.norm(back - want) <= 2.0 ** -8 * np.linalg.norm(want) * 1.01


# ---- gemm -------------------------------------------------------------------

def check_gemm(m, n, k, dtype, bias, tile, lo=118, hi=134, fill=0):
    rng = np.random.default_rng(m * 7 + n + k + tile)
    xc, xs, xv = held(rng, m, k, lo, hi, fill)
    wc, ws, wv = held(rng, n, k, lo, hi, fill)
    b = dev(rng.standard_normal(n) * 50, dtype) if bias else None
    y = f64(cr.convrot_gemm_mx4(xc, xs, wc, ws, b, dtype=dtype, tile=tile))
    want, mass = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    if bias:
        want, mass = want + f64(b), mass + np.abs(f64(b))
    half, tiny = H16[dtype]
    tol = (half + 2 * U) * np.abs(want) + tiny + (k + 1) * U * mass
    inside = np.abs(want) + tol < MAX16[dtype]
    assert (np.abs(y - want)[inside] <= tol[inside]).all()


@pytest.mark.parametrize("dtype,bias", [(torch.bfloat16, False), (torch.float16, True)],
                         ids=["bf16", "f16-bias"])
@pytest.mark.parametrize("m,n,k", [
    (1, 16, 32), (1, 48, 256), (2, 400, 96), (9, 208, 3840), (16, 64, 288), (17, 112, 512),
    (33, 80, 1056), (64, 16, 5120), (65, 16, 64), (65, 144, 288), (100, 272, 32),
    (129, 400, 544), (300, 208, 1280), (257, 528, 224)])
def test_gemm_matches_oracle(m, n, k, dtype, bias):
    check_gemm(m, n, k, dtype, bias, 0, lo=118 if dtype == torch.bfloat16 else 121,
               hi=134 if dtype == torch.bfloat16 else 128, fill=255)


@pytest.mark.parametrize("tile", [16, 64, 128, 192, 256, 384])
@pytest.mark.parametrize("n,k", [(16, 32), (416, 256), (592, 800), (208, 2272)])
def test_gemm_forced_variants(tile, n, k):
    for m in ((1, 11, 16, 17, 32, 33, 64) if tile == 16 else
              (1, tile // 2 + 3, tile, tile + 1, 2 * tile + 37)):
        check_gemm(m, n, k, torch.bfloat16, True, tile)


@pytest.mark.parametrize("m", [5, 30, 64])
def test_gemm_few_rows_at_every_block_width(m):
    """Blocks of 16, 32 and 64 columns: fewer compute units make them wider."""
    rng = np.random.default_rng(m)
    xc, xs, _ = held(rng, m, 1056)
    wc, ws, _ = held(rng, 432, 1056)
    want = cr.convrot_gemm_mx4(xc, xs, wc, ws, tile=16)
    widths = set()
    try:
        for cus in (256, 24, 12, 7, 1):
            cr.convrot_set_compute_units(cus)
            if cr.convrot_plan_launch("gemm_mx4", m=m, n=432, k=1056)["tile_m"] == 16:
                widths.add(cr.convrot_plan_launch("gemm_mx4", m=m, n=432, k=1056)["tile_n"])
            assert torch.equal(cr.convrot_gemm_mx4(xc, xs, wc, ws, tile=16), want), cus
    finally:
        cr.convrot_set_compute_units(0)
    assert len(widths) >= 2
    check_gemm(m, 432, 1056, torch.bfloat16, True, 16)


@pytest.mark.parametrize("m", [3, 40, 130, 700])
@pytest.mark.parametrize("k", [96, 1024, 4352])
def test_gemm_is_exact_where_fp32_is(m, k):
    """One scale for all: every sum is a multiple of 1/4 below 2^22 in any order,
    so y is the exact sum rounded once."""
    rng = np.random.default_rng(m + k)
    n = 272
    xc, xs, xv = held(rng, m, k, 127, 128)
    wc, ws, wv = held(rng, n, k, 127, 128)
    for dtype in DTYPES:
        y = cr.convrot_gemm_mx4(xc, xs, wc, ws, dtype=dtype).cpu()
        want = torch.from_numpy(xv @ wv.T).to(torch.float32).to(dtype)
        assert torch.equal(y, want)
    # every tiled variant gives the same bits
    if m > 64:
        for tile in (64, 128, 192, 256, 384):
            assert torch.equal(cr.convrot_gemm_mx4(xc, xs, wc, ws, dtype=dtype, tile=tile).cpu(),
                               want)


def test_gemm_scales_at_the_ends_of_the_range():
    """2^-127 against 2^127 is 1; 2^-127 twice underflows to zero."""
    rng = np.random.default_rng(11)
    for m in (5, 200):
        xc, xs, xv = held(rng, m, 512, 0, 1)
        wc, ws, wv = held(rng, 32, 512, 254, 255)
        y = cr.convrot_gemm_mx4(xc, xs, wc, ws, dtype=torch.float16).cpu()
        want = torch.from_numpy(xv @ wv.T).to(torch.float32).to(torch.float16)
        assert torch.equal(y, want)
        ws.zero_()
        assert (cr.convrot_gemm_mx4(xc, xs, wc, ws) == 0).all()


def test_gemm_writes_nothing_beside_y():
    rng = np.random.default_rng(12)
    for m, n in ((3, 48), (130, 144)):
        xc, xs, _ = held(rng, m, 320)
        wc, ws, _ = held(rng, n, 320)
        buf = torch.full((m + 2, n), 3.0, dtype=torch.bfloat16, device=DEV)
        cr.convrot_gemm_mx4(xc, xs, wc, ws, out=buf[1:m + 1])
        assert (buf[0] == 3.0).all() and (buf[m + 1] == 3.0).all()
        assert torch.equal(buf[1:m + 1], cr.convrot_gemm_mx4(xc, xs, wc, ws))


def test_gemm_operand_offsets_behind_4_gib():
    """y rows behind 2^32 bytes: a tall x (codes shared by stride-free repeats)."""
    rng = np.random.default_rng(13)
    m, n, k = 70000, 32768, 32
    xc, xs, xv = held(rng, 16, k, 125, 129)
    wc, ws, wv = held(rng, n, k, 125, 129)
    big_c = xc.repeat(m // 16, 1)
    big_s = xs.repeat(1, m // 16, 1)
    y = cr.convrot_gemm_mx4(big_c, big_s, wc, ws)
    want = torch.from_numpy(xv @ wv.T).to(torch.float32).to(torch.bfloat16)
    for r in (0, 32768, 65520, m - 16):
        assert torch.equal(y[r:r + 16].cpu(), want)


# ---- linear -----------------------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f16"])
@pytest.mark.parametrize("g,m,n,k", [(1, 5, 32, 96), (4, 70, 48, 128), (16, 1, 160, 288),
                                     (64, 65, 144, 576), (256, 1, 3840, 3840),
                                     (256, 9, 400, 1024), (256, 200, 272, 768)])
def test_linear_is_quantize_then_gemm(g, m, n, k, dtype):
    rng = np.random.default_rng(m + n + k)
    x = dev(tokens(rng, m, k), dtype)
    w = dev(rng.standard_normal((n, k)) * 0.02, torch.bfloat16)
    b = dev(rng.standard_normal(n), dtype)
    wc, ws = cr.convrot_quantize_mx4(w, g, SEED)
    y = cr.convrot_linear_mx4(x, wc, ws, g, SEED, b)
    want = cr.convrot_gemm_mx4(*cr.convrot_quantize_mx4(x, g, SEED), wc, ws, b, dtype=dtype)
    assert torch.equal(y, want)


def test_linear_does_not_depend_on_slices():
    rng = np.random.default_rng(21)
    m, n, k, g = 700, 272, 768, 256
    x = dev(tokens(rng, m, k), torch.bfloat16)
    wc, ws = cr.convrot_quantize_mx4(dev(rng.standard_normal((n, k)), torch.bfloat16), g, SEED)
    want = cr.convrot_linear_mx4(x, wc, ws, g, SEED)
    assert torch.equal(want, cr.convrot_gemm_mx4(*cr.convrot_quantize_mx4(x, g, SEED), wc, ws))
    for rows in (1, 15, 64, 300, 699):
        size = cr.convrot_linear_mx4_workspace_for_rows(rows, k)
        pad = torch.full((size + 256,), 91, dtype=torch.uint8, device=DEV)
        out = cr.convrot_linear_mx4(x, wc, ws, g, SEED, workspace=pad[:size])
        assert torch.equal(out, want), rows
        assert (pad[size:] == 91).all(), rows
    x = x[:40]
    want = cr.convrot_linear_mx4(x, wc, ws, g, SEED)
    for rows in (1, 7, 33):
        size = cr.convrot_linear_mx4_workspace_for_rows(rows, k)
        pad = torch.empty(size, dtype=torch.uint8, device=DEV)
        assert torch.equal(cr.convrot_linear_mx4(x, wc, ws, g, SEED, workspace=pad), want), rows


def test_no_rows():
    for g in (1, 256):
        x = torch.empty((0, 256), dtype=torch.bfloat16, device=DEV)
        c, s = cr.convrot_quantize_mx4(x, g, SEED)
        assert c.shape == (0, 128) and s.shape == (1, 0, 8)
        assert cr.convrot_dequant_mx4(c, s, g).shape == (0, 256)
        w = cr.convrot_quantize_mx4(torch.ones((16, 256), dtype=torch.bfloat16, device=DEV), g)
        assert cr.convrot_gemm_mx4(c, s, *w).shape == (0, 16)
        assert cr.convrot_linear_mx4(x, *w, g).shape == (0, 16)


def test_streams_and_graph_replays_equal_eager():
    """Calls on a side stream, and a captured step replayed with eager work and
    synchronizations in between."""
    rng = np.random.default_rng(31)
    g, k, n = 256, 1024, 528
    wc, ws = cr.convrot_quantize_mx4(dev(rng.standard_normal((n, k)), torch.bfloat16), g, SEED)
    xs = [dev(tokens(rng, m, k), torch.bfloat16) for m in (1, 40, 300)]
    want = [cr.convrot_linear_mx4(x, wc, ws, g, SEED) for x in xs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [cr.convrot_linear_mx4(x, wc, ws, g, SEED) for x in xs]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [cr.convrot_linear_mx4(x, wc, ws, g, SEED) for x in xs]
    for rep in range(4):
        for x, o in zip(xs, outs):
            x.copy_(x.flip(0))
            o.zero_()
        want = [cr.convrot_linear_mx4(x, wc, ws, g, SEED) for x in xs]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), rep


def test_gemm_bits_do_not_depend_on_the_tile():
    """Sums that fp32 rounds: the tiled variants add in the same order."""
    rng = np.random.default_rng(41)
    xc, xs, _ = held(rng, 500, 2144, 110, 140)
    wc, ws, _ = held(rng, 432, 2144, 110, 140)
    want = cr.convrot_gemm_mx4(xc, xs, wc, ws)
    for tile in (64, 128, 192, 256, 384):
        assert torch.equal(cr.convrot_gemm_mx4(xc, xs, wc, ws, tile=tile), want), tile
    # ... nor on the compute units, automatic choice included
    try:
        for cus in (256, 128, 3):
            cr.convrot_set_compute_units(cus)
            assert torch.equal(cr.convrot_gemm_mx4(xc, xs, wc, ws), want), cus
            for m in (1, 20, 50):
                part = (xc[:m], xs[:, :-(-m // 16) * 16].contiguous())
                got = cr.convrot_gemm_mx4(*part, wc, ws)
                cr.convrot_set_compute_units(256)
                assert torch.equal(cr.convrot_gemm_mx4(*part, wc, ws), got), (cus, m)
                cr.convrot_set_compute_units(cus)
    finally:
        cr.convrot_set_compute_units(0)


@pytest.mark.parametrize("tile,bm", [(40, 64), (96, 64), (160, 128)])
@pytest.mark.parametrize("n,k", [(16, 32), (416, 256), (592, 800), (208, 2272)])
def test_gemm_rectangular_tiles(tile, bm, n, k):
    for m in (1, bm // 2 + 3, bm, bm + 1, 2 * bm + 37):
        check_gemm(m, n, k, torch.bfloat16, True, tile)


@pytest.mark.parametrize("m,n,k", [(129, 144, 32), (300, 400, 544), (700, 272, 4352)])
def test_gemm_128_tiles_one_and_two_to_a_cu(m, n, k):
    """A grid of up to one tile per CU takes the longer copy ring; the bits agree."""
    rng = np.random.default_rng(m)
    xc, xs, _ = held(rng, m, k, 110, 140)
    wc, ws, _ = held(rng, n, k, 110, 140)
    want = cr.convrot_gemm_mx4(xc, xs, wc, ws, tile=256)
    try:
        for cus in (256, 1):
            cr.convrot_set_compute_units(cus)
            for tile in (40, 96, 128, 160):
                assert torch.equal(cr.convrot_gemm_mx4(xc, xs, wc, ws, tile=tile), want), (cus, tile)
            check_gemm(m, n, k, torch.float16, True, 128, lo=121, hi=128)
    finally:
        cr.convrot_set_compute_units(0)


# ---- offsets that pass 32 bits ------------------------------------------------
# A tensor of 63 rows over and over: 63 and the powers of two that an offset could
# wrap by have no common factor, so a wrapped row is another row.

LONG = 131072                # the longest row
FOLD = 63


def folded(rows, times):
    """A [63, ...] tensor `times` times over."""
    return rows.repeat(times, *[1] * (rows.dim() - 1))


def folded_scales(scales, times):
    """Scales of 63 rows, likewise, in their own layout."""
    held_rows = scales[:, :FOLD].repeat(1, times, 1)
    pad = torch.zeros((scales.shape[0], -held_rows.shape[1] % 16, 8), dtype=torch.uint8, device=DEV)
    return torch.cat([held_rows, pad], 1)


def test_quantize_and_dequant_behind_4_gib():
    """x and out of 8.7e9 elements, codes of 4.3 GB."""
    rng = np.random.default_rng(51)
    g, times = 256, 1050
    base = dev(tokens(rng, FOLD, LONG), torch.bfloat16)
    want_c, want_s = cr.convrot_quantize_mx4(base, g, SEED)
    want = cr.convrot_dequant_mx4(want_c, want_s, g, SEED)
    assert_quantized(want_c[:4], want_s, f64(base[:4]), g)
    x = folded(base, times)
    codes, scales = cr.convrot_quantize_mx4(x, g, SEED)
    del x
    assert codes.numel() > 1 << 32
    assert (codes.view(times, FOLD, -1) == want_c).all()
    assert torch.equal(scales[:, :FOLD * times], folded_scales(want_s, times)[:, :FOLD * times])
    out = cr.convrot_dequant_mx4(codes, scales, g, SEED)
    assert (out.view(times, FOLD, -1) == want).all()


@pytest.mark.parametrize("side", ["x", "w"])
def test_gemm_codes_behind_4_gib(side):
    """Codes of 4.3 GB on either side, in the tiled kernel and the one for few
    rows; one scale for all, so that y is the exact sum rounded once: multiples of
    1/4 whose partial sums stay below 2^22."""
    rng = np.random.default_rng(52)
    times = 1056
    bc, bs, bv = held(rng, FOLD, LONG, 127, 128)
    big_c, big_s = folded(bc, times), folded_scales(bs, times)
    assert big_c.numel() > 1 << 32
    for rows in (16,) if side == "x" else (4, 80):
        oc, os_, ov = held(rng, rows, LONG, 127, 128)
        for tile in (0, 64, 256, 384) if side == "x" or rows > 64 else (0, 16):
            if side == "x":
                y = cr.convrot_gemm_mx4(big_c, big_s, oc, os_, tile=tile)
                y = y.view(times, FOLD, rows)
                want = bv @ ov.T
            else:
                y = cr.convrot_gemm_mx4(oc, os_, big_c, big_s, tile=tile)
                y = y.view(rows, times, FOLD).transpose(0, 1)
                want = ov @ bv.T
            want = torch.from_numpy(want).to(torch.float32).to(torch.bfloat16).to(DEV)
            assert (y == want).all(), (rows, tile)
