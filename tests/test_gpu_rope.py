"""GPU: rotary tables, and norms of q and k with the rotation, against a float64
oracle.

Bounds (u = 2^-24). A table entry is one rounding of cos or sin of a float64 angle,
which itself is off by a few 2^-52 of its size. A norm is off by 64 u of each value
(sums are trees of at most 8 + 6 + 16 + 16 additions of squares off by u, their root and
products a few roundings more), a layer norm also by the mean's error, 49 u of the mean
of |v| over its deviation; the weight's product adds u, the rotation u of either product
and of the sum; then one rounding to 16 bits."""

import numpy as np
import pytest
import torch

import int8_gemm_amd as cr
from oracle import attention_ref as ref
from oracle import mx4_ref

pytestmark = pytest.mark.gpu

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
    return t.detach().cpu().to(torch.float64).numpy()


def table_close(got, positions, dims, theta, shared):
    ang = ref.angles(positions, dims, theta, shared)
    for i, want in ((0, np.cos(ang)), (1, np.sin(ang))):
        tol = U * np.abs(want) + 16 * 2.0 ** -52 * (1 + np.abs(ang))
        assert (np.abs(f64(got)[..., i] - want) <= tol).all()


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64, torch.float32])
@pytest.mark.parametrize("tokens,dims,theta,shared", [
    (1, (128,), 10000.0, False), (7, (2,), 256.0, False), (33, (16, 56, 56), 10000.0, False),
    (16, (44, 42, 42), 10000.0, True), (17, (32, 48, 48), 256.0, True),
    (1000, (6, 10, 2, 4), 5e5, False), (129, (256,), 1e6, False), (5, (2,) * 8, 0.5, True)])
def test_table(tokens, dims, theta, shared, dtype):
    rng = np.random.default_rng(tokens)
    pos = rng.integers(-1000, 100000, (tokens, len(dims)))
    if dtype == torch.float32:
        pos = pos / 8.0
    got = cr.convrot_rope_table(dev(pos, dtype), dims, theta, shared=shared)
    assert got.shape == (tokens, sum(dims) // 2, 2) and got.dtype == torch.float32
    table_close(got, pos, dims, theta, shared)


def test_table_far_positions_strides_and_out():
    pos = np.array([0, 1, 2 ** 20, 2 ** 31 - 1, -2 ** 31, 2 ** 40, -2 ** 45])
    table_close(cr.convrot_rope_table(dev(pos, torch.int64), [64]), pos, (64,), 10000.0, False)
    # axes as rows of one tensor, every second token of it
    wide = np.arange(3 * 40).reshape(3, 40) * 7
    at = dev(wide, torch.int32)[:, ::2].t()
    out = torch.full((20, 6, 2), 9.0, device=DEV)
    assert cr.convrot_rope_table(at, (4, 4, 4), out=out) is out
    table_close(out, wide[:, ::2].T, (4, 4, 4), 10000.0, False)
    # one position for all, and no tokens
    same = dev(np.array([[5, 6]]), torch.int64).expand(9, 2)
    table_close(cr.convrot_rope_table(same, (4, 8)), np.tile([[5, 6]], (9, 1)), (4, 8), 10000.0,
                False)
    assert cr.convrot_rope_table(same[:0], (4, 8)).shape == (0, 6, 2)
    nan = cr.convrot_rope_table(dev(np.array([np.nan, np.inf, 1.0]), torch.float32), [4])
    assert torch.isnan(nan[:2]).all() and torch.isfinite(nan[2]).all()


def norm_and_error(v, kind, weight):
    if kind is None:
        return v, 0 * v
    y = mx4_ref.norm(v, kind, None, EPS)
    err = 64 * U * np.abs(y)
    if kind == "layer":
        std = np.sqrt(v.var(-1, keepdims=True) + EPS)
        err = err + 49 * U * np.abs(v).mean(-1, keepdims=True) / std
    if weight is not None:
        y, err = y * weight, (err + U * np.abs(y)) * np.abs(weight)
    return y, err


def heads_close(got, x, norm, span, weight, table, halves):
    half, tiny = H16[got.dtype]
    t, h, d = x.shape
    v = f64(x)
    w = None if weight is None else f64(weight).reshape(-1)
    if span == "row":
        y, err = norm_and_error(v.reshape(t, h * d), norm, w)
        y, err = y.reshape(t, h, d), err.reshape(t, h, d)
    else:
        y, err = norm_and_error(v, norm, w)
    if table is not None:
        tab = np.tile(f64(table), (t // table.shape[0], 1, 1))
        # sizes of the terms: |a c| + |b s|, and the same of their errors
        size = np.abs(tab) * [1, -1]
        mag, err = ref.rotate(np.abs(y), size, halves), ref.rotate(err, size, halves)
        flip = np.abs(tab)
        mag2, err2 = ref.rotate(np.abs(y), flip, halves), ref.rotate(err, flip, halves)
        mag, err = np.maximum(np.abs(mag), np.abs(mag2)), np.maximum(np.abs(err), np.abs(err2))
        y = ref.rotate(y, tab, halves)
        err = err + 2 * U * mag
    tol = (half + 2 * U) * np.abs(y) + tiny + err * (1 + half)
    bad = np.abs(f64(got) - y) > tol
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[0])


def make(rng, t, hq, hk, d, pairs, norm, span, weights, dtype):
    qkv = dev(rng.standard_normal((t, hq + 2 * hk, d)) * 3 + 0.5, dtype)
    kw = {"norm": norm, "span": span}
    if weights and norm:
        n = (hq * d, hk * d) if span == "row" else (d, d)
        kw["q_weight"] = dev(1 + 0.2 * rng.standard_normal(n[0]), dtype)
        kw["k_weight"] = dev(1 + 0.2 * rng.standard_normal(n[1]), dtype)
    table = None
    if pairs:
        ang = rng.uniform(-1000, 1000, (t, pairs))
        table = dev(np.stack([np.cos(ang), np.sin(ang)], -1), torch.float32)
    return qkv[:, :hq], qkv[:, hq:hq + hk], table, kw


def check(q, k, table, kw, halves, got):
    for x, y, w in ((q, got[0], "q_weight"), (k, got[1], "k_weight")):
        heads_close(y, x, kw["norm"], kw["span"], kw.get(w), table, halves)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("norm,span", [("rms", "head"), ("layer", "head"), ("rms", "row"),
                                       ("layer", "row"), (None, "head")])
@pytest.mark.parametrize("t,hq,hk,d,pairs,halves", [
    (1, 1, 1, 8, 4, False), (1, 32, 8, 128, 64, True), (5, 3, 1, 16, 8, True),
    (67, 24, 8, 64, 16, True), (33, 30, 30, 128, 64, False), (9, 5, 5, 72, 36, False),
    (9, 5, 5, 72, 32, True), (7, 40, 2, 128, 48, False), (3, 80, 10, 256, 128, True),
    (4, 65, 1, 96, 0, False), (130, 2, 1, 40, 12, False), (11, 1, 7, 24, 8, True),
    (2, 128, 128, 256, 128, False), (6, 9, 3, 8, 0, True)])
def test_heads_match_oracle(t, hq, hk, d, pairs, halves, norm, span, dtype):
    rng = np.random.default_rng(t + d)
    for weights in (True, False):
        q, k, table, kw = make(rng, t, hq, hk, d, pairs, norm, span, weights, dtype)
        got = cr.convrot_qk_norm_rope(q, k, table, halves=halves, eps=EPS, **kw)
        assert got[0].shape == q.shape and got[1].shape == k.shape and got[0].is_contiguous()
        check(q, k, table, kw, halves, got)


@pytest.mark.parametrize("span", ["head", "row"])
@pytest.mark.parametrize("halves", [False, True])
def test_in_place_in_a_fused_projection(span, halves):
    rng = np.random.default_rng(5)
    for t in (1, 37):
        q, k, table, kw = make(rng, t, 12, 4, 64, 32, "rms", span, True, torch.bfloat16)
        whole = q._base if q._base is not None else q
        before = whole.clone()
        want = cr.convrot_qk_norm_rope(q, k, table, halves=halves, **kw)
        got = cr.convrot_qk_norm_rope(q, k, table, halves=halves, q_out=q, k_out=k, **kw)
        assert got[0] is q and got[1] is k
        assert torch.equal(q, want[0]) and torch.equal(k, want[1])
        assert torch.equal(whole[:, 16:], before[:, 16:])      # v


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("halves", [False, True], ids=["neighbours", "halves"])
@pytest.mark.parametrize("heads,d,pairs", [(3, 64, 8), (3, 64, 16), (1, 128, 24), (5, 72, 32),
                                           (40, 128, 40), (2, 256, 64), (2, 40, 16)])
def test_elements_behind_the_pairs_stay(heads, d, pairs, halves, dtype):
    """Without a norm they are what they were, infinities, NaN and the sign of a zero too,
    whatever lies beside them."""
    rng = np.random.default_rng(d + pairs)
    tokens = 70
    x = rng.standard_normal((tokens, heads, d))
    tail = x[..., 2 * pairs:]
    kind = rng.integers(0, 6, tail.shape)
    for i, what in enumerate((np.inf, -np.inf, np.nan, -0.0, 0.0)):
        tail[kind == i] = what
    q = dev(x, dtype)
    angle = rng.random((tokens, pairs)) * 6
    table = dev(np.stack((np.cos(angle), np.sin(angle)), -1), torch.float32)
    got, _ = cr.convrot_qk_norm_rope(q, table=table, norm=None, halves=halves)
    want = ref.rotate(f64(q)[..., :2 * pairs], f64(table), halves)
    head = f64(got)[..., :2 * pairs]
    assert (np.abs(head - want) <= H16[dtype][0] * np.abs(want) + 8 * U * np.abs(x).max(
        where=np.isfinite(x), initial=0)).all()
    a, b = (t[..., 2 * pairs:].contiguous() for t in (got, q))
    some = ~b.isnan()
    assert torch.equal(a[some].view(torch.int16), b[some].view(torch.int16))
    assert a[~some].isnan().all()


def test_other_layouts():
    rng = np.random.default_rng(6)
    dt, t, h, d = torch.bfloat16, 20, 6, 64
    # heads that interleave q, k and v, in place; a head-major layout; two of four sequences
    mix = dev(rng.standard_normal((t, h, 3, d)), dt)
    q, k, v = (mix[:, :, i] for i in range(3))
    ang = rng.uniform(-9, 9, (t, d // 2))
    table = dev(np.stack([np.cos(ang), np.sin(ang)], -1), torch.float32)
    q0, k0, v0 = q.clone(), k.clone(), v.clone()
    cr.convrot_qk_norm_rope(q, k, table, q_out=q, k_out=k)
    check(q0, k0, table, {"norm": "rms", "span": "head"}, False, (q, k))
    assert torch.equal(v, v0)
    major = dev(rng.standard_normal((h, t, d)), dt).transpose(0, 1)
    out = torch.zeros((h, t, d), dtype=dt, device=DEV).transpose(0, 1)
    got, none = cr.convrot_qk_norm_rope(major, None, table, norm="layer", q_out=out)
    assert got is out and none is None
    heads_close(out, major, "layer", "head", None, table, False)
    # a batch shares the table; new keys go straight into rows of a cache
    x = dev(rng.standard_normal((2, t, h, d)), dt)
    cache = torch.full((2, t, 3 * h, d), 7.0, dtype=dt, device=DEV)
    qb, _ = cr.convrot_qk_norm_rope(x, x[:, :, :2], table, k_out=cache[:, :, 4:6])
    heads_close(qb.reshape(2 * t, h, d), x.reshape(2 * t, h, d), "rms", "head", None, table, False)
    assert torch.equal(cache[:, :, 4:6], qb[:, :, :2]) and (cache[:, :, :4] == 7).all()
    assert (cache[:, :, 6:] == 7).all()
    # no tokens
    a, b = cr.convrot_qk_norm_rope(q[:0], k[:0], None)
    assert a.shape == (0, h, d) and b.shape == (0, h, d)


@pytest.mark.parametrize("span", ["head", "row"])
@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_rows_of_any_magnitude(norm, span):
    """bf16 reaches 2^-133 and 2^127, whose squares fp32 does not hold; ordinary heads
    beside such ones keep their bits."""
    rng = np.random.default_rng(7)
    t, h, d = 40, 4, 64
    base = rng.standard_normal((t, h, d))
    plain = dev(base, torch.bfloat16)
    x = plain.clone()
    powers = np.linspace(-120, 124, 20).astype(int)
    x[::2] = (x[::2].double() * torch.from_numpy(2.0 ** powers).to(DEV)[:, None, None]).bfloat16()
    got, _ = cr.convrot_qk_norm_rope(x, None, None, norm=norm, span=span, eps=0.0)
    want, _ = cr.convrot_qk_norm_rope(plain, None, None, norm=norm, span=span, eps=0.0)
    assert torch.equal(got[1::2], want[1::2])
    v = f64(x[::2]) / (2.0 ** powers)[:, None, None]     # the norm does not see the power
    v = v.reshape(20, h * d) if span == "row" else v
    y = mx4_ref.norm(v, norm, None, 0.0).reshape(20, h, d)
    err = 64 * U * np.abs(y) + (49 * U if norm == "layer" else 0)
    assert (np.abs(f64(got[::2]) - y) <= 2.0 ** -8 * np.abs(y) + err * 1.01 + 2.0 ** -134).all()
    zero, _ = cr.convrot_qk_norm_rope(torch.zeros_like(x), None, None, norm=norm, span=span)
    assert (zero == 0).all()


def test_runs_streams_and_graphs():
    rng = np.random.default_rng(8)
    q, k, table, kw = make(rng, 333, 24, 8, 64, 32, "rms", "row", True, torch.float16)
    pos = dev(np.arange(333 * 3).reshape(333, 3), torch.int64)
    want = cr.convrot_qk_norm_rope(q, k, table, **kw)
    want_t = cr.convrot_rope_table(pos, (16, 24, 24))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = cr.convrot_qk_norm_rope(q, k, table, **kw)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out = [torch.zeros_like(t) for t in (*want, want_t)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cr.convrot_rope_table(pos, (16, 24, 24), out=out[2])
        cr.convrot_qk_norm_rope(q, k, table, q_out=out[0], k_out=out[1], **kw)
    for _ in range(3):
        for t in out:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, (*want, want_t)))
        torch.ones(1000, device=DEV).sum().item()


def test_offsets_beyond_32_bits():
    """Rows past 2^31 elements: the bits of the same rows in a call of their own."""
    dt, h, d, last = torch.bfloat16, 2, 128, 37
    rng = np.random.default_rng(5)
    # a table of 2^32 entries
    t = (1 << 24) + 5
    pos = torch.arange(t, dtype=torch.int32, device=DEV)
    table = cr.convrot_rope_table(pos, (256,))
    want = cr.convrot_rope_table(pos[-last:], (256,))
    assert torch.equal(table[-last:], want)
    del table
    # tokens of a wide tensor, in place, and next to it
    n = 1100
    wide = torch.empty((n, 1 << 21), dtype=dt, device=DEV)
    q, k = (wide[:, i * h * d:(i + 1) * h * d].view(n, h, d) for i in range(2))
    x = dev(rng.standard_normal((2, n, h, d)), dt)
    q.copy_(x[0])
    k.copy_(x[1])
    turns = cr.convrot_rope_table(pos[:n], (128,))
    for span in ("head", "row"):
        want = cr.convrot_qk_norm_rope(x[0], x[1], turns, span=span)
        got = cr.convrot_qk_norm_rope(q, k, turns, span=span)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    cr.convrot_qk_norm_rope(q, k, turns, span="row", q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    del wide, q, k
    # more rows than a 32-bit count of elements holds, the table's rows in turn
    n = (1 << 19) * 20
    x = torch.empty((n, h, d), dtype=dt, device=DEV)
    x[:1000] = 0
    x[-last:] = dev(rng.standard_normal((last, h, d)), dt)
    got, _ = cr.convrot_qk_norm_rope(x, None, turns[:1024])
    rows = torch.arange(n - last, n, device=DEV) % 1024
    want, _ = cr.convrot_qk_norm_rope(x[-last:], None, turns[rows])
    assert torch.equal(got[-last:], want)
