"""GPU: the gated residual norm against a float64 oracle.

Bounds: the sums over a row are trees of at most 32 + 6 + 8 additions, so a sum
of K terms is off by at most 46 u sum|terms| (u = 2^-24); mean square and its
root add a few roundings more, counted as 64 u relative in all. A layer norm's
mean is off by at most 48 u mean|v|, which enters each element as it is. x' and
h are then rounded once to 16 bits. h is compared with the oracle's norm of the
x' that the kernel returned, as the contract says."""

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
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    cr.load_library()


def dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).to(DEV)


def f64(t):
    return t.cpu().to(torch.float64).numpy()


def norm_and_error(v, kind, weight):
    """The norm, and how far fp32 may be off before the weight's own roundings."""
    y = ref.norm(v, kind, None, EPS)
    err = 64 * U * np.abs(y)
    if kind == "layer":
        std = np.sqrt(v.var(-1, keepdims=True) + EPS)
        err = err + 49 * U * np.abs(v).mean(-1, keepdims=True) / std
    if weight is not None:
        y, err = y * weight, (err + U * np.abs(y)) * np.abs(weight)
    return y, err


def check(x, o, x_out, h, kw):
    dtype, m = x.dtype, x.shape[0]
    half, tiny = H16[dtype]
    mod = {n: None if kw.get(n) is None else ref.per_row(f64(kw[n]), m)
           for n in ("gate", "scale", "shift")}
    opt = {n: None if kw.get(n) is None else f64(kw[n]) for n in ("weight", "post_weight")}
    if o is not None:
        t, err = f64(o), 0.0
        if kw.get("post_norm"):
            t, err = norm_and_error(t, kw["post_norm"], opt["post_weight"])
        if mod["gate"] is not None:
            t, err = t * mod["gate"], (err + U * np.abs(t)) * np.abs(mod["gate"])
        want = f64(x) + t
        tol = (half + 2 * U) * np.abs(want) + tiny + err
        assert (np.abs(f64(x_out) - want) <= tol).all()
    y, err = norm_and_error(f64(x_out), kw.get("norm", "rms"), opt["weight"])
    if mod["scale"] is not None:
        s = 1 + mod["scale"]
        y, err = y * s, err * np.abs(s) + 3 * U * np.abs(y * s)
    if mod["shift"] is not None:
        y, err = y + mod["shift"], err + 2 * U * (np.abs(y) + np.abs(mod["shift"]))
    # a row of one value has layer norm 0 / sqrt(eps): the mean's error is all there is
    tol = (half + 2 * U) * np.abs(y) + tiny + err * (1 + half)
    assert (np.abs(f64(h) - y) <= tol).all()


def build(rng, m, k, dtype, samples, post, weights, mods, residual=True):
    x = dev(rng.standard_normal((m, k)) * 3 + 0.5, dtype)
    o = dev(rng.standard_normal((m, k)) * 2, dtype) if residual else None
    kw = {}
    if post and residual:
        kw["post_norm"] = post
        if weights:
            kw["post_weight"] = dev(1 + 0.2 * rng.standard_normal(k), dtype)
    if weights:
        kw["weight"] = dev(1 + 0.2 * rng.standard_normal(k), dtype)
    if mods:
        wide = dev(0.5 * rng.standard_normal((samples, 6 * k)), dtype)
        if residual:
            kw["gate"] = wide[:, 2 * k:3 * k]
        kw["shift"], kw["scale"] = wide[:, 3 * k:4 * k], wide[:, 4 * k:5 * k]
    return x, o, kw


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("norm,post", [("rms", "rms"), ("layer", None), ("rms", "layer"),
                                       ("layer", "rms")])
@pytest.mark.parametrize("m,k,samples", [(1, 8, 1), (67, 256, 1), (3, 264, 3), (36, 512, 4),
                                         (10, 1024, 2), (9, 1032, 1), (6, 2048, 3),
                                         (5, 2056, 1), (4, 3840, 2), (3, 5120, 1), (2, 16384, 2)])
def test_norm_residual_matches_oracle(m, k, samples, norm, post, dtype):
    rng = np.random.default_rng(m + k)
    for weights, mods in ((True, True), (False, True), (True, False), (False, False)):
        x, o, kw = build(rng, m, k, dtype, samples, post, weights, mods)
        x_out, h = cr.convrot_norm_residual(x, o, norm=norm, eps=EPS, **kw)
        check(x, o, x_out, h, {**kw, "norm": norm})
    # no residual: x itself is normed and returned
    x, _, kw = build(rng, m, k, dtype, samples, None, True, True, residual=False)
    x_out, h = cr.convrot_norm_residual(x, norm=norm, eps=EPS, **kw)
    assert x_out is x
    check(x, None, x, h, {**kw, "norm": norm})


def test_rows_of_one_value_of_zeros_and_with_a_far_mean():
    rng = np.random.default_rng(1)
    k = 3840
    x = np.zeros((4, k))
    x[1] = 5.0
    x[2] = 1000 + rng.standard_normal(k)
    x[3] = rng.standard_normal(k) * 1e-20
    t = dev(x, torch.bfloat16)
    for norm in ("rms", "layer"):
        x_out, h = cr.convrot_norm_residual(t, norm=norm)
        check(t, None, x_out, h, {"norm": norm})
        assert (h[0] == 0).all()
    assert (cr.convrot_norm_residual(t, norm="layer")[1][1] == 0).all()


def test_not_finite_rows_stay_to_themselves():
    rng = np.random.default_rng(2)
    for k in (256, 5120):
        x = rng.standard_normal((9, k))
        o = rng.standard_normal((9, k))
        x[2, 5], o[4, k - 1], x[6, 0] = np.nan, np.inf, -np.inf
        x, o = dev(x, torch.bfloat16), dev(o, torch.bfloat16)
        x_out, h = cr.convrot_norm_residual(x, o, norm="rms", post_norm=None)
        clean = [r for r in range(9) if r not in (2, 4, 6)]
        assert torch.isfinite(h[clean]).all() and torch.isfinite(x_out[clean]).all()
        assert torch.isnan(h[2]).all() and torch.isnan(h[4, k - 1]) and torch.isnan(h[6, 0])
        check(x[clean], o[clean], x_out[clean], h[clean], {})


def test_in_place_and_given_buffers():
    rng = np.random.default_rng(3)
    x, o, kw = build(rng, 12, 1288, torch.bfloat16, 3, "rms", True, True)
    want = cr.convrot_norm_residual(x, o, **kw)
    buf = torch.full((14, 1288), 9.0, dtype=torch.bfloat16, device=DEV)
    y = x.clone()
    x_out, h = cr.convrot_norm_residual(y, o, x_out=y, h=buf[1:13], **kw)
    assert x_out is y and torch.equal(y, want[0]) and torch.equal(buf[1:13], want[1])
    assert (buf[0] == 9.0).all() and (buf[13] == 9.0).all()


def test_modulation_rows_of_any_stride():
    rng = np.random.default_rng(4)
    m, k = 8, 512
    x, o, _ = build(rng, m, k, torch.float16, 1, None, False, False)
    one = dev(rng.standard_normal(k), torch.float16)
    many = dev(rng.standard_normal((4, k)), torch.float16)
    per_token = dev(rng.standard_normal((m, k)), torch.float16)
    for kw in ({"gate": one, "scale": many}, {"gate": many, "scale": one[None], "shift": one},
               {"scale": many.repeat(1, 2)[:, k:], "shift": many},
               {"gate": per_token, "shift": per_token}):
        x_out, h = cr.convrot_norm_residual(x, o, norm="layer", **kw)
        check(x, o, x_out, h, {**kw, "norm": "layer"})


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("g,m,k", [(1, 3, 96), (4, 5, 288), (16, 2, 2080), (64, 9, 1088),
                                   (256, 1, 256), (256, 41, 256), (64, 19, 512), (16, 5, 1024),
                                   (256, 6, 3840), (256, 3, 16384)])
def test_quantized_h_is_the_16_bit_h_quantized(g, m, k, dtype):
    rng = np.random.default_rng(g + k)
    x, o, kw = build(rng, m, k, dtype, 1, "rms", True, True)
    x_out, h = cr.convrot_norm_residual(x, o, **kw)
    want = cr.convrot_quantize_mx4(h, g, SEED)
    also = torch.zeros_like(x)
    scales = torch.full_like(want[1], 55)
    got = cr.convrot_norm_residual_mx4(x, o, g, SEED, h=also, scales=scales, **kw)
    assert torch.equal(got[0], x_out) and torch.equal(also, h)
    assert torch.equal(got[1], want[0])
    assert torch.equal(got[2][:, :m], want[1][:, :m]) and (scales[:, m:] == 55).all()
    # without the 16-bit h the same
    again = cr.convrot_norm_residual_mx4(x, o, g, SEED, **kw)
    assert torch.equal(again[1], want[0])


def test_last_sample_may_be_short():
    """The C call: row r takes modulation row r / rows_per_mod, here 4, 4 and 2 rows."""
    import ctypes

    from int8_gemm_amd import mx4
    rng = np.random.default_rng(8)
    m, k = 10, 264
    x = dev(rng.standard_normal((m, k)), torch.float16)
    scale = dev(rng.standard_normal((3, 2 * k)), torch.float16)
    h = torch.empty_like(x)
    a = mx4._NormArgs(x=x.data_ptr(), h=h.data_ptr(), m=m, k=k, rows_per_mod=4, norm=1, dtype=1,
                      eps=EPS, scale=scale.data_ptr(), scale_stride=2 * k)
    stream = torch.cuda.current_stream().cuda_stream
    assert cr.load_library().convrot_norm_residual(ctypes.byref(a), stream) == 0
    full = scale[[0, 0, 0, 0, 1, 1, 1, 1, 2, 2], :k]
    check(x, None, x, h, {"scale": full})


def test_a_block_of_layers_captured_and_replayed():
    """Two blocks as a model would run them: norm into 4 bits, projection, gated
    residual and norm into the next projection; graph replays equal eager runs,
    which equal the unfused calls."""
    rng = np.random.default_rng(9)
    m, k, n, g = 200, 768, 768, 256
    dt = torch.bfloat16
    ws = [cr.convrot_quantize_mx4(dev(rng.standard_normal((n, k)) * 0.05, dt), g, SEED)
          for _ in range(2)]
    mod = dev(0.3 * rng.standard_normal((2, 6 * k)), dt)
    weight = dev(1 + 0.1 * rng.standard_normal(k), dt)
    x = dev(rng.standard_normal((m, k)), dt)
    cut = [mod[:, i * k:(i + 1) * k] for i in range(6)]

    def fused():
        _, c, s = cr.convrot_norm_residual_mx4(x, None, g, SEED, weight=weight, scale=cut[0],
                                               shift=cut[1])
        y = cr.convrot_gemm_mx4(c, s, *ws[0])
        x1, c, s = cr.convrot_norm_residual_mx4(x, y, g, SEED, gate=cut[2], post_norm="rms",
                                                post_weight=weight, norm="layer", scale=cut[3],
                                                shift=cut[4])
        y = cr.convrot_gemm_mx4(c, s, *ws[1])
        return cr.convrot_norm_residual(x1, y, gate=cut[5])

    def unfused():
        _, h = cr.convrot_norm_residual(x, weight=weight, scale=cut[0], shift=cut[1])
        y = cr.convrot_linear_mx4(h, *ws[0], g, SEED)
        x1, h = cr.convrot_norm_residual(x, y, gate=cut[2], post_norm="rms", post_weight=weight,
                                         norm="layer", scale=cut[3], shift=cut[4])
        y = cr.convrot_linear_mx4(h, *ws[1], g, SEED)
        return cr.convrot_norm_residual(x1, y, gate=cut[5])

    want = unfused()
    assert all(torch.equal(a, b) for a, b in zip(fused(), want))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = fused()
    for rep in range(4):
        x.copy_(x.flip(0))
        want = unfused()
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), rep


def test_grids_that_fill_the_card_give_the_same_bits():
    """Rows beyond what the CUs hold at once take a form with fewer registers; a
    card of one CU takes it for a few rows already."""
    rng = np.random.default_rng(12)
    for k in (1024, 5120):
        x, o, kw = build(rng, 24, k, torch.bfloat16, 2, "layer", True, True)
        want = cr.convrot_norm_residual(x, o, **kw)
        quantized = cr.convrot_norm_residual_mx4(x, o, 256, SEED, **kw)
        try:
            cr.convrot_set_compute_units(1)
            got = cr.convrot_norm_residual(x, o, **kw)
            again = cr.convrot_norm_residual_mx4(x, o, 256, SEED, **kw)
        finally:
            cr.convrot_set_compute_units(0)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        check(x, o, got[0], got[1], kw)
        assert torch.equal(again[1], quantized[1])
        assert torch.equal(again[2][:, :24], quantized[2][:, :24])


def test_no_rows():
    x = torch.empty((0, 256), dtype=torch.bfloat16, device=DEV)
    x_out, h = cr.convrot_norm_residual(x, torch.empty_like(x))
    assert h.shape == (0, 256)
    assert cr.convrot_norm_residual_mx4(x, None, 256)[1].shape == (0, 128)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_sign_of_zero(dtype):
    """-0 + -0 is -0 in x', and the norm keeps the sign; -0 + 0 is 0."""
    x = dev(np.full((3, 64), -0.0), dtype)
    o = x.clone()
    o[:, ::2] = 0.0
    x_out, h = cr.convrot_norm_residual(x, o)
    want = torch.zeros(64, dtype=torch.bool)
    want[1::2] = True
    for t in (x_out, h):
        assert (t == 0).all()
        assert torch.equal(torch.signbit(t).cpu(), want.expand(3, 64))


def check_norm(x, h, kind, eps):
    """h against the norm of x with this eps; the bounds of the file's head, which hold
    for any magnitude (a row's power of two is taken out of it before it is squared)."""
    v, eps = f64(x), float(np.float32(eps))
    y = ref.norm(v, kind, None, eps)
    half, tiny = H16[x.dtype]
    err = 64 * U * np.abs(y)
    if kind == "layer":
        err = err + 49 * U * np.abs(v).mean(-1, keepdims=True) \
            / np.sqrt(v.var(-1, keepdims=True) + eps)
    assert (np.abs(f64(h) - y) <= (half + 2 * U) * np.abs(y) + tiny + err * (1 + half)).all()


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("k", [8, 256, 520, 1024, 3840, 16384])
def test_rows_of_every_magnitude(k, norm):
    """bf16 rows whose squares leave the range of fp32 at either end, beside ordinary
    rows of the same wave, which keep their bits; one large element; the largest
    and smallest values of the format."""
    rng = np.random.default_rng(k)
    x = rng.standard_normal((24, k)) + 0.25
    for r, e in enumerate((-132, -125, -100, -80, -60, -45, 40, 60, 64, 90, 120, 124)):
        x[2 * r] *= 2.0 ** e
    x[1] = np.where(rng.random(k) < 0.5, 1, -1) * float(torch.finfo(torch.bfloat16).max)
    x[3] = 2.0 ** -133 * rng.integers(1, 4, k)
    x[5, 3] = 1e30
    x[7, 3] = -3e38
    t = dev(x, torch.bfloat16)
    plain = [9, 11, 13, 15, 17, 19, 21, 23]
    for eps in (1e-6, 0.0, 1e-38, 1e-30, 1e30, 3e38):
        _, h = cr.convrot_norm_residual(t, norm=norm, eps=eps)
        assert torch.isfinite(h).all()
        check_norm(t, h, norm, eps)
        _, alone = cr.convrot_norm_residual(t[plain].contiguous(), norm=norm, eps=eps)
        assert torch.equal(h[plain], alone)


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("k", [512, 5120])
def test_post_norms_of_every_magnitude_and_in_place(k, norm):
    """The same for o, with x' written over x, and for an x' that is large itself;
    the quantized h is the 16-bit h quantized."""
    rng = np.random.default_rng(k + 1)
    x = rng.standard_normal((8, k))
    o = rng.standard_normal((8, k)) * np.exp2([[-130], [-90], [-50], [0], [50], [70], [100], [125]])
    x[1] *= 2.0 ** 100
    o, t = dev(o, torch.bfloat16), dev(x, torch.bfloat16)
    given = t.clone()
    for eps in (0.0, 1e-6):
        y, h = cr.convrot_norm_residual(t, o, post_norm=norm, norm=norm, eps=eps)
        post = torch.zeros_like(t)
        check_norm(o, cr.convrot_norm_residual(o, norm=norm, eps=eps)[1], norm, eps)
        cr.convrot_norm_residual(post, o, post_norm=norm, x_out=post, norm=norm, eps=eps)
        check_norm(o, post, norm, eps)      # 0 + post(o)
        check_norm(y, h, norm, eps)
        out, also = cr.convrot_norm_residual(given, o, post_norm=norm, x_out=given, norm=norm,
                                             eps=eps)
        assert torch.equal(out, y) and torch.equal(also, h)
        given.copy_(t)
        _, codes, scales = cr.convrot_norm_residual_mx4(t, o, 256, SEED, post_norm=norm, norm=norm,
                                                        eps=eps)
        want = cr.convrot_quantize_mx4(h, 256, SEED)
        assert torch.equal(codes, want[0]) and torch.equal(scales[:, :8], want[1][:, :8])


def test_rows_of_zeros_without_eps():
    """0 / sqrt(0): NaN, in the row of zeros alone."""
    x = torch.ones((5, 64), dtype=torch.bfloat16, device=DEV)
    x[2] = 0
    h = cr.convrot_norm_residual(x, eps=0.0)[1]
    assert torch.isnan(h[2]).all() and (h[[0, 1, 3, 4]] == 1).all()


def test_rows_per_mod_beyond_the_rows():
    """The C call: any rows_per_mod of at least m is one modulation row for all."""
    import ctypes

    from int8_gemm_amd import mx4
    rng = np.random.default_rng(18)
    m, k = 10, 264
    x = dev(rng.standard_normal((m, k)), torch.bfloat16)
    shift = dev(rng.standard_normal((3, k)), torch.bfloat16)
    want = cr.convrot_norm_residual(x, shift=shift[0], eps=EPS)[1]
    for rows in (m, m + 1, 2 ** 32 + 1, 2 ** 63 - 1):
        h = torch.zeros_like(x)
        a = mx4._NormArgs(x=x.data_ptr(), h=h.data_ptr(), m=m, k=k, rows_per_mod=rows, norm=1,
                          eps=EPS, shift=shift.data_ptr(), shift_stride=k)
        stream = torch.cuda.current_stream().cuda_stream
        assert cr.load_library().convrot_norm_residual(ctypes.byref(a), stream) == 0
        assert torch.equal(h, want), rows


def test_rows_behind_2_to_the_31_elements():
    """63 rows over and over (a wrapped offset would meet another row); x' in place."""
    rng = np.random.default_rng(21)
    fold, times, k, g = 63, 2100, 16384, 64
    x, o, kw = build(rng, fold, k, torch.bfloat16, 1, "rms", True, True)
    want_x, want_c, want_s = cr.convrot_norm_residual_mx4(x, o, g, SEED, **kw)
    want_h = cr.convrot_norm_residual(x, o, **kw)[1]
    check(x, o, want_x, want_h, kw)
    big, o = x.repeat(times, 1), o.repeat(times, 1)
    assert big.numel() > 1 << 31
    h = torch.empty_like(big)
    out, codes, scales = cr.convrot_norm_residual_mx4(big, o, g, SEED, x_out=big, h=h, **kw)
    for got, want in ((out, want_x), (h, want_h), (codes, want_c)):
        assert (got.view(times, fold, -1) == want).all()
    assert torch.equal(scales[:, :fold * times], want_s[:, :fold].repeat(1, times, 1))
