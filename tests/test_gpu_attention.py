"""GPU: attention over packed sequences against a float64 oracle.

Bounds (u = 2^-24, A = the mean of |v| under a row's softmax weights, S = sum |q k| of a
score, N keys): a score is off by (d + 8) 2 u S scale; the exponent's argument and its
multiply-adds by 4 u of the largest |scaled score|, the power of two by 4 u, the running
maximum's factors by 4 u a tile. Relative errors e of the weights move the output by at
most 2 e A. The weights' rounding to 16 bits adds h A (h = 2^-8 bf16, 2^-11 half; half
weights below 2^-14 of the largest are off by 2^-25 of it, N times that against a sum of
at least 1), the sums of N terms 2 N u A. Then one rounding of the output."""

import math

import numpy as np
import pytest
import torch

import int8_gemm_amd as cr
from oracle import attention_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
H16 = {torch.bfloat16: (2.0 ** -8, 2.0 ** -134), torch.float16: (2.0 ** -11, 2.0 ** -25)}
DTYPES = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])


@pytest.fixture(scope="module", autouse=True)
def _lib():
    cr.load_library()


def dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).to(DEV)


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def offsets(lens):
    return torch.tensor([0, *np.cumsum(lens)], dtype=torch.int32, device=DEV)


def close(q, k, v, out, lse, scale, causal):
    """One sequence's results against the oracle's."""
    dtype = out.dtype
    half, tiny = H16[dtype]
    q, k, v = f64(q), f64(k), f64(v)
    n, hq, d = q.shape
    length, hk, _ = k.shape
    want, want_lse, spread = ref.attention(q, k, v, scale, causal)
    kk = np.repeat(k, hq // hk, 1)
    # the largest sum of |q k| and the largest score of a row
    size = np.abs(q).max(-1) * np.abs(kk).sum(-1).max(0, initial=0.0)[None]
    if length:
        size = np.minimum(size, np.sqrt((q ** 2).sum(-1) * (kk ** 2).sum(-1).max(0)[None]))
    e = (d + 8) * 2 * U * size * scale + 4 * U * size * scale + 4 * U + 4 * U * (length / 32 + 2)
    top = np.abs(v).max() if v.size else 0.0
    tol = (2 * e[..., None] + half + 4 * length * U) * spread
    if dtype == torch.float16:
        tol = tol + length * 2.0 ** -25 * top
    tol = tol * 1.01 + (half + 2 * U) * np.abs(want) + tiny
    bad = ~(np.abs(f64(out) - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[0].tolist())
    if lse is not None:
        got = f64(lse)
        none = want_lse == -np.inf
        assert (got[none] == -np.inf).all()
        got, want_lse = np.where(none, 0, got), np.where(none, 0, want_lse)
        err = (e.T + (length + 8) * U + 4 * U * np.abs(want_lse))
        assert (np.abs(got - want_lse) <= err).all()


def make(rng, q_lens, k_lens, hq, hk, d, dtype, heat=1.0):
    q = dev(rng.standard_normal((sum(q_lens), hq, d)) * heat, dtype)
    k = dev(rng.standard_normal((sum(k_lens), hk, d)), dtype)
    v = dev(rng.standard_normal((sum(k_lens), hk, d)), dtype)
    return q, k, v


def run_packed(q, k, v, q_lens, k_lens, causal, **kw):
    out, lse = cr.convrot_attention(q, k, v, q_offsets=offsets(q_lens),
                                    k_offsets=offsets(k_lens), causal=causal, return_lse=True, **kw)
    return out, lse


def check_packed(q, k, v, out, lse, q_lens, k_lens, causal, scale=None):
    scale = scale or 1 / math.sqrt(q.shape[-1])
    qo, ko = np.cumsum([0, *q_lens]), np.cumsum([0, *k_lens])
    for b in range(len(q_lens)):
        qs, ks = slice(qo[b], qo[b + 1]), slice(ko[b], ko[b + 1])
        close(q[qs], k[ks], v[ks], out[qs], lse[:, qs], scale, causal)


LENS = [
    ([1], [1]), ([1], [63]), ([1], [64]), ([5], [65]), ([33], [33]), ([129], [200]),
    ([200], [129]), ([1, 0, 7, 130, 64], [1, 5, 0, 130, 31]), ([257, 3], [300, 1000]),
    ([0, 0], [4, 0]), ([1, 1, 1], [700, 1, 4097]), ([513], [513])]


@DTYPES
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("q_lens,k_lens", LENS)
@pytest.mark.parametrize("hq,hk,d", [(2, 2, 128), (6, 2, 64), (8, 1, 128)])
def test_lengths(q_lens, k_lens, hq, hk, d, causal, dtype):
    rng = np.random.default_rng(sum(q_lens) + 7 * sum(k_lens))
    q, k, v = make(rng, q_lens, k_lens, hq, hk, d, dtype, 3.0)
    out, lse = run_packed(q, k, v, q_lens, k_lens, causal)
    check_packed(q, k, v, out, lse, q_lens, k_lens, causal)


@DTYPES
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("tile,hq,hk,d", [(256, 2, 2, 128), (256, 6, 2, 72), (256, 8, 1, 96),
                                          (32, 3, 1, 128), (32, 4, 2, 64), (32, 2, 2, 256),
                                          (128, 4, 1, 128), (128, 2, 1, 256)])
@pytest.mark.parametrize("q_lens,k_lens", [([1], [64]), ([300], [300]), ([129], [200]),
                                           ([200], [129]), ([1, 0, 7, 530, 64], [1, 5, 0, 530, 31]),
                                           ([257, 3], [300, 1000]), ([600], [1500]),
                                           ([40, 700], [2000, 90]), ([3, 2], [65, 193])])
def test_each_kernel(q_lens, k_lens, tile, hq, hk, d, causal, dtype):
    """The kernels that sizes choose from, at sizes that would choose another."""
    rng = np.random.default_rng(sum(q_lens) + tile)
    q, k, v = make(rng, q_lens, k_lens, hq, hk, d, dtype, 3.0)
    out, lse = run_packed(q, k, v, q_lens, k_lens, causal, tile=tile)
    check_packed(q, k, v, out, lse, q_lens, k_lens, causal)


@DTYPES
@pytest.mark.parametrize("tile,hq,hk,d", [(256, 4, 2, 128), (128, 4, 2, 128), (32, 4, 2, 128),
                                          (128, 3, 1, 64), (128, 1, 1, 256)])
def test_scores_that_climb_and_fall(tile, hq, hk, d, dtype):
    """Keys whose scores rise from tile to tile move every row's reference many times;
    falling ones never do; both with rows beside them that see other keys."""
    rng = np.random.default_rng(d + tile)
    n, length = 300, 700
    q, k, v = make(rng, [n], [length], hq, hk, d, dtype, 0.3)
    slope = torch.linspace(-1, 1, length, device=DEV)[:, None, None] * 40 / d ** 0.5
    for sign in (1, -1):
        qs = (q.float() + 1).to(dtype)
        ks = (k.float() * 0.3 + sign * slope).to(dtype)
        for causal in (False, True):
            out, lse = cr.convrot_attention(qs, ks, v, causal=causal, return_lse=True, tile=tile)
            close(qs, ks, v, out, lse, d ** -0.5, causal)


# every kernel: the two of many rows, that of few, heads of each padded size
EACH = [(256, 4, 2, 128), (128, 4, 2, 128), (32, 4, 2, 128), (128, 3, 1, 64), (32, 3, 1, 64),
        (128, 1, 1, 256), (32, 2, 1, 256), (256, 2, 2, 96)]


@pytest.mark.parametrize("tile,hq,hk,d", EACH)
@pytest.mark.parametrize("power", [90, 97, 120])
def test_large_values_under_scores_that_climb_and_fall(tile, hq, hk, d, power):
    """Scores that climb by 31 octaves behind a row's first keys, and values of which fp32
    does not hold 2^31 times as much; a column of small ones beside them, and one of an
    infinity."""
    rng = np.random.default_rng(d + tile)
    n, length = 300, 700
    q, k, v = make(rng, [n], [length], hq, hk, d, torch.bfloat16, 0.3)
    level = np.interp(np.arange(length), [0, 100, 350, 500, length], [0, 0, 31, 31, 0])
    q[:, :, 0] = 1
    k[:, :, 0] = dev(level * math.log(2) * d ** 0.5, torch.bfloat16)[:, None]
    v *= 2.0 ** power
    v[:, :, 1] *= 2.0 ** (-60 - power)
    for causal in (False, True):
        out, lse = cr.convrot_attention(q, k, v, causal=causal, return_lse=True, tile=tile)
        close(q, k, v, out, lse, d ** -0.5, causal)
        one = v.clone()
        one[600, :, 5] = math.inf
        got, got_lse = cr.convrot_attention(q, k, one, causal=causal, return_lse=True, tile=tile)
        sees = torch.arange(n, device=DEV) + length - n >= (600 if causal else 0)
        assert (got[sees][:, :, 5] == math.inf).all()
        got[sees, :, 5] = out[sees, :, 5]
        assert torch.equal(got, out) and torch.equal(got_lse, lse)


@pytest.mark.parametrize("tile,hq,hk,d", EACH)
@pytest.mark.parametrize("n,length", [(300, 700), (2, 9000), (40, 5000)])
def test_values_whose_sum_leaves_fp32(n, length, tile, hq, hk, d):
    """Equal scores and values of nearly the largest bf16: their mean is one, their sum is
    not; one block's keys and parts that are joined."""
    rng = np.random.default_rng(n)
    q, k, v = make(rng, [n], [length], hq, hk, d, torch.bfloat16)
    k[:] = k[:1]
    v = dev((1.25 + 0.5 * rng.random((length, hk, d))) * 2.0 ** 127, torch.bfloat16)
    v[:, :, ::3] *= -1
    for causal in (False, True):
        out, lse = cr.convrot_attention(q, k, v, causal=causal, return_lse=True, tile=tile)
        close(q, k, v, out, lse, d ** -0.5, causal)


@DTYPES
@pytest.mark.parametrize("tile,hq,hk,d", EACH)
@pytest.mark.parametrize("levels", [(-1e6,), (-1e9, -1e5), (-1e30,)], ids=str)
def test_keys_far_below_the_others_take_no_bits_from_them(tile, hq, hk, d, levels, dtype):
    """A row's first keys may score any distance below those that carry its weight: the
    tolerance is that of the latter alone. Some rows score all keys alike, others by half."""
    if dtype == torch.float16:
        levels = [max(x, -6e4) for x in levels]     # of half's range, times q and scale
    rng = np.random.default_rng(d + tile)
    n, length, far = 300, 900, 160
    q, k, v = make(rng, [n], [length], hq, hk, d, dtype, 2.0)
    scale = d ** -0.5
    up = 1.0 if dtype == torch.bfloat16 else 64.0
    q[:, :, 0] = dev(rng.choice([0, 0.5, 1], (n, hq)) * up, dtype)
    q[:, 0, 0] = up
    k[:, :, 0] = 0
    each = far // len(levels)
    for i, x in enumerate(levels):
        k[i * each:(i + 1) * each, :, 0] = x if dtype == torch.float16 else x / scale
    v[:far] = 100
    for causal in (False, True):
        out, lse = cr.convrot_attention(q, k, v, causal=causal, return_lse=True, tile=tile)
        for h in range(hq):
            low = (q[:, h, 0] > 0).cpu()
            g = h // (hq // hk)
            qh, kh, vh = q[:, h:h + 1], k[:, g:g + 1], v[:, g:g + 1]
            rest, kh = qh.clone(), kh.clone()
            rest[:, :, 0] = kh[:, :, 0] = 0         # 0 on one side or both where a key counts
            for rows, keys in ((low, (kh[far:], vh[far:])), (~low, (kh, vh))):
                if not causal:
                    close(rest[rows], *keys, out[rows, h:h + 1], lse[h:h + 1, rows], scale, False)
                elif rows.all():
                    close(rest, *keys, out[:, h:h + 1], lse[h:h + 1], scale, True)


@DTYPES
@pytest.mark.parametrize("tile,hq,hk,d", EACH)
@pytest.mark.parametrize("n,length", [(300, 500), (3, 6000), (40, 33)])
def test_rows_all_of_whose_keys_score_far_below_zero(n, length, tile, hq, hk, d, dtype):
    """The softmax does not know how far; heads and rows of different distance side by side."""
    rng = np.random.default_rng(d + tile + n)
    q, k, v = make(rng, [n], [length], hq, hk, d, dtype, 2.0)
    scale = d ** -0.5
    q[:, :, 0] = dev(rng.choice([0, 0.75, 1, 1.25, 2, 30], (n, hq)), dtype)
    k[:, :, 0] = -177.4 / scale                 # about 2^-256, and further
    for causal in (False, True):
        out, lse = cr.convrot_attention(q, k, v, causal=causal, return_lse=True, tile=tile)
        close(q, k, v, out, lse, scale, causal)


@DTYPES
@pytest.mark.parametrize("tile,hq,hk,d", EACH)
@pytest.mark.parametrize("level", [-120, -160, -192, -224, -256, -288])
def test_keys_a_little_below_the_others_far_below_zero(level, tile, hq, hk, d, dtype):
    """First keys 2 and 6 octaves below the others, all of them `level` octaves below one."""
    rng = np.random.default_rng(d + tile - level)
    n, length = 290, 450
    q, k, v = make(rng, [n], [length], hq, hk, d, dtype, 0.1)
    q[:, :, 0] = 1
    octaves = level + np.where(np.arange(length) < 97, -6, np.where(np.arange(length) < 225, -2, 0))
    k[:, :, 0] = dev(octaves * math.log(2) * d ** 0.5, dtype)[:, None]
    v[:225] += 4
    for causal in (False, True):
        out, lse = cr.convrot_attention(q, k, v, causal=causal, return_lse=True, tile=tile)
        close(q, k, v, out, lse, d ** -0.5, causal)


@DTYPES
@pytest.mark.parametrize("tile,hq,hk,d", EACH + [(128, 4, 2, 72), (128, 3, 1, 40)])
@pytest.mark.parametrize("n,length", [(300, 500), (9, 6000)])
def test_rows_beside_one_that_is_formed_again_keep_their_bits(n, length, tile, hq, hk, d, dtype):
    rng = np.random.default_rng(d + tile + n)
    q, k, v = make(rng, [n], [length], hq, hk, d, dtype, 4.0)
    k[:, :, 0] = -2000
    q[:, :, 0] = 0
    for causal in (False, True):
        want, want_lse = cr.convrot_attention(q, k, v, causal=causal, return_lse=True, tile=tile)
        other = q.clone()
        other[7, :, 0] = 16                     # scores of -4000 and less
        got, lse = cr.convrot_attention(other, k, v, causal=causal, return_lse=True, tile=tile)
        rest = [i for i in range(n) if i != 7]
        assert torch.equal(got[rest], want[rest]) and torch.equal(lse[:, rest], want_lse[:, rest])
        assert (lse[:, 7] < -1000).all()


@DTYPES
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("hq,hk,d", [(1, 1, 8), (3, 3, 16), (4, 2, 40), (5, 1, 64), (2, 1, 72),
                                     (4, 4, 80), (3, 1, 96), (2, 2, 112), (7, 1, 128),
                                     (2, 1, 136), (3, 3, 192), (4, 2, 256)])
def test_heads(hq, hk, d, causal, dtype):
    rng = np.random.default_rng(d)
    q_lens, k_lens = [37, 150, 1], [37, 211, 90]
    q, k, v = make(rng, q_lens, k_lens, hq, hk, d, dtype, 2.0)
    out, lse = run_packed(q, k, v, q_lens, k_lens, causal)
    check_packed(q, k, v, out, lse, q_lens, k_lens, causal)


@DTYPES
@pytest.mark.parametrize("hq,hk,d,n,length", [(3, 3, 128, 1100, 1300), (2, 1, 64, 2100, 900),
                                              (2, 2, 256, 300, 700), (24, 8, 128, 9, 20000),
                                              (4, 4, 96, 77, 5000)])
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
def test_larger(hq, hk, d, n, length, causal, dtype):
    rng = np.random.default_rng(n)
    q, k, v = make(rng, [n], [length], hq, hk, d, dtype, 4.0)
    out, lse = cr.convrot_attention(q, k, v, causal=causal, return_lse=True)
    close(q, k, v, out, lse, 1 / math.sqrt(d), causal)


@DTYPES
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("hq,hk,d,lens,tile", [
    (4, 4, 128, [700, 65], 0), (8, 2, 64, [1, 300, 33], 0), (2, 1, 256, [200, 5], 0),
    (4, 1, 72, [130, 64], 0), (4, 4, 128, [700, 65], 256), (4, 1, 72, [130, 64], 256),
    (4, 4, 128, [300, 65], 32)])
def test_each_query_finds_its_key(hq, hk, d, lens, tile, causal, dtype):
    """Scores that leave one key: the output is that key's value, to the bit."""
    rng = np.random.default_rng(d)
    q, k, v = make(rng, lens, lens, hq, hk, d, dtype)
    k = torch.sign(k) * 2                        # any two differ in many signs
    at = np.concatenate([rng.integers(0, np.arange(1, n + 1) if causal else n, n)
                         + sum(lens[:i]) for i, n in enumerate(lens)])
    at = torch.from_numpy(at).to(DEV)
    q = (torch.sign(k)[at] * 4).repeat_interleave(hq // hk, 1)
    out, _ = run_packed(q, k, v, lens, lens, causal, scale=8.0, tile=tile)
    # equal keys share the weight: drop queries whose key comes again
    for h in range(hq):
        kh = k[:, h // (hq // hk)].float()
        sc = q[:, h].float() @ kh.t()
        seq = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(lens)).to(DEV)
        sc[seq[:, None] != seq[None]] = -math.inf
        best = sc.topk(min(2, sc.shape[1]), 1).values
        alone = best[:, 0] - best[:, -1] >= 16       # 16 * 8 in the exponent: e^-128
        assert alone.float().mean() > 0.5
        assert torch.equal(out[alone, h], v[at[alone], h // (hq // hk)])


@DTYPES
@pytest.mark.parametrize("batch,hq,hk,d,room", [(1, 8, 2, 128, 9000), (12, 8, 2, 128, 2000),
                                                (70, 4, 1, 64, 700), (200, 2, 1, 64, 300),
                                                (5, 6, 3, 256, 3000), (1030, 1, 1, 64, 200)])
def test_single_tokens_over_caches_of_different_use(batch, hq, hk, d, room, dtype):
    rng = np.random.default_rng(batch)
    used = rng.integers(0, room + 1, batch)
    used[0], used[-1] = room, 1 if batch > 1 else room
    q = dev(rng.standard_normal((batch, 1, hq, d)) * 2, dtype)
    k = dev(rng.standard_normal((batch, room, hk, d)), dtype)
    v = dev(rng.standard_normal((batch, room, hk, d)), dtype)
    lens = torch.from_numpy(used).to(torch.int32).to(DEV)
    out, lse = cr.convrot_attention(q, k, v, k_lens=lens, causal=True, return_lse=True)
    # the same packed, by offsets
    flat = [torch.cat([t[b, :n] for b, n in enumerate(used)]) for t in (k, v)]
    packed, packed_lse = cr.convrot_attention(q[:, 0], *flat, q_offsets=offsets([1] * batch),
                                              k_offsets=offsets(used), return_lse=True)
    some = range(batch) if batch <= 70 else [0, 1, 63, 64, 65, 127, 128, batch - 2, batch - 1]
    for b in some:
        n = int(used[b])
        close(q[b], k[b, :n], v[b, :n], out[b], lse[:, b:b + 1], d ** -0.5, True)
        close(q[b], k[b, :n], v[b, :n], packed[b:b + 1], packed_lse[:, b:b + 1], d ** -0.5, True)
    assert (packed - out[:, 0]).abs().max() <= 2 * H16[dtype][0] * 8


@DTYPES
def test_a_padded_cache_and_what_it_holds_behind_its_use(dtype):
    rng = np.random.default_rng(3)
    batch, room, hq, hk, d = 5, 300, 8, 2, 128
    lens = [300, 1, 0, 131, 64]
    q = dev(rng.standard_normal((batch, 2, hq, d)) * 2, dtype)
    k = dev(rng.standard_normal((batch, room, hk, d)), dtype)
    v = dev(rng.standard_normal((batch, room, hk, d)), dtype)
    k[2, :] = math.nan
    for b, n in enumerate(lens):
        k[b, n:] = math.nan
        v[b, n:] = math.inf
    used = torch.tensor(lens, dtype=torch.int32, device=DEV)
    for causal in (False, True):
        out, lse = cr.convrot_attention(q, k, v, k_lens=used, causal=causal, return_lse=True)
        assert out.shape == q.shape
        for b, n in enumerate(lens):
            close(q[b], k[b, :n], v[b, :n], out[b], lse[:, 2 * b:2 * b + 2], 1 / math.sqrt(d),
                  causal)
    # more than there is room for, and less than nothing
    wild = torch.tensor([1 << 30, -5, 0, 131, 64], dtype=torch.int32, device=DEV)
    k, v = torch.nan_to_num(k, 0.0), torch.nan_to_num(v, 0.0, 0.0, 0.0)
    out = cr.convrot_attention(q, k, v, k_lens=wild)
    close(q[0], k[0], v[0], out[0], None, 1 / math.sqrt(d), False)
    assert (out[1] == 0).all() and (out[2] == 0).all()


@DTYPES
@pytest.mark.parametrize("hq,hk,d,n,length,tile", [
    (2, 2, 128, 200, 200, 0), (4, 1, 64, 90, 300, 0), (2, 1, 256, 70, 70, 0),
    (8, 1, 128, 2, 3000, 0), (3, 3, 40, 300, 100, 0), (2, 2, 128, 600, 600, 256),
    (4, 2, 96, 300, 500, 256), (2, 2, 128, 200, 200, 32)])
@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
def test_keys_that_the_mask_hides_have_no_part(hq, hk, d, n, length, tile, what, dtype):
    """Non-finite keys and values: queries that do not see them are what they are
    without them, the others get what they get from them."""
    rng = np.random.default_rng(n)
    q, k, v = make(rng, [n], [length], hq, hk, d, dtype)
    clean = cr.convrot_attention(q, k, v, causal=True, tile=tile)
    at = length - 1 - min(length, n) // 2      # seen by the later queries only
    col = d - 3
    v[at, :, col] = what
    got = cr.convrot_attention(q, k, v, causal=True, tile=tile)
    sees = torch.arange(n, device=DEV) + length - n >= at
    assert torch.equal(got[~sees], clean[~sees])
    hit = got[sees][:, :, col]
    assert (torch.isnan(hit) if math.isnan(what) else hit == what).all()
    rest = [c for c in range(d) if c != col]
    assert torch.equal(got[sees][:, :, rest], clean[sees][:, :, rest])
    # two of opposite sign meet
    if math.isinf(what) and at + 1 < length:
        v[at + 1, :, col] = -what
        got = cr.convrot_attention(q, k, v, causal=True, tile=tile)
        both = torch.arange(n, device=DEV) + length - n >= at + 1
        assert torch.isnan(got[both][:, :, col]).all()
        assert (got[sees & ~both][:, :, col] == what).all()
    # a key: its scores are hidden as well
    v[:, :, col] = 0
    clean = cr.convrot_attention(q, k, v, causal=True, tile=tile)
    k[at] = what
    got = cr.convrot_attention(q, k, v, causal=True, tile=tile)
    assert torch.equal(got[~sees], clean[~sees])


@DTYPES
@pytest.mark.parametrize("tile,hq,hk,d", [
    (256, 4, 2, 72), (256, 2, 2, 96), (256, 2, 1, 128), (128, 4, 2, 80), (128, 2, 2, 120),
    (128, 3, 1, 8), (128, 3, 1, 40), (128, 1, 1, 64), (128, 1, 1, 136), (128, 2, 1, 192),
    (128, 1, 1, 256), (32, 4, 2, 72), (32, 3, 1, 40), (32, 2, 1, 160), (32, 2, 1, 128)])
def test_an_infinite_key_that_is_seen(tile, hq, hk, d, dtype):
    """A score of -infinity has no weight, wherever in the head the infinity stands; one of
    +infinity leaves no result."""
    rng = np.random.default_rng(d)
    n, length, at = 300, 500, 77
    q, k, v = make(rng, [n], [length], hq, hk, d, dtype)
    keep = [j for j in range(length) if j != at]
    for col in (d - 1, d - 8, 0):
        q[:, :, col] = q[:, :, col].abs() + 0.125
        x = k.clone()
        x[at, :, col] = -math.inf
        out, lse = cr.convrot_attention(q, x, v, return_lse=True, tile=tile)
        close(q, k[keep], v[keep], out, lse, d ** -0.5, False)
        # causal rows all see it
        out, lse = cr.convrot_attention(q, x, v, causal=True, return_lse=True, tile=tile)
        close(q, k[keep], v[keep], out, lse, d ** -0.5, True)
        x[at, :, col] = math.inf
        out, lse = cr.convrot_attention(q, x, v, return_lse=True, tile=tile)
        assert out.isnan().all() and not lse.isfinite().any()


@DTYPES
@pytest.mark.parametrize("hq,hk,d,n,length,tile", [
    (2, 2, 128, 200, 70, 128), (4, 2, 64, 90, 300, 0), (2, 1, 256, 70, 129, 0),
    (2, 2, 128, 3, 33, 32),
    (2, 2, 128, 600, 100, 256), (4, 2, 96, 300, 3001, 256), (3, 3, 40, 300, 64, 0),
    (1, 1, 128, 100, 4097, 128)])
@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
def test_the_last_key_of_a_tile_that_ends_early(hq, hk, d, n, length, tile, what, dtype):
    """The places behind it hold nothing, whatever its value is."""
    rng = np.random.default_rng(length)
    q, k, v = make(rng, [n], [length], hq, hk, d, dtype)
    clean = cr.convrot_attention(q, k, v, tile=tile)
    col = d - 3
    v[length - 1, :, col] = what
    got = cr.convrot_attention(q, k, v, tile=tile)
    hit = got[:, :, col]
    assert (torch.isnan(hit) if math.isnan(what) else hit == what).all()
    rest = [c for c in range(d) if c != col]
    assert torch.equal(got[:, :, rest], clean[:, :, rest])


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("n,d,tile", [(1, 128, 0), (5, 64, 0), (300, 128, 0), (300, 128, 256),
                                      (300, 128, 128), (70, 256, 0), (70, 64, 32)])
def test_no_keys(n, d, tile, causal):
    q = torch.ones((n, 4, d), dtype=torch.bfloat16, device=DEV)
    none = q[:0, :2]
    for args in ({}, {"q_offsets": offsets([n]), "k_offsets": offsets([0])}):
        out, lse = cr.convrot_attention(q, none, none, causal=causal, tile=tile,
                                        return_lse=True, **args)
        assert not out.any() and (lse == -math.inf).all()
    k = torch.full((200, 2, d), math.nan, dtype=torch.bfloat16, device=DEV)
    used = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = cr.convrot_attention(q, k, k, k_lens=used, causal=causal, tile=tile,
                                    return_lse=True)
    assert not out.any() and (lse == -math.inf).all()
    assert cr.convrot_attention(q[:0], k, k, causal=causal, tile=tile).shape == (0, 4, d)


@DTYPES
def test_many_heads(dtype):
    rng = np.random.default_rng(13)
    q, k, v = make(rng, [3], [50], 1000, 500, 8, dtype)
    close(q, k, v, *cr.convrot_attention(q, k, v, causal=True, return_lse=True), 8 ** -0.5, True)


def test_rows_outside_the_sequences_stay():
    rng = np.random.default_rng(4)
    hq, hk, d = 4, 2, 64
    for splits_len in (40, 5000):            # the second is split over the keys
        q, k, v = make(rng, [50], [splits_len], hq, hk, d, torch.bfloat16)
        out = torch.full_like(q, 7.0)
        lse = torch.full((hq, 50), 7.0, device=DEV)
        qo = torch.tensor([3, 13, 40], dtype=torch.int32, device=DEV)
        ko = torch.tensor([0, 9, splits_len], dtype=torch.int32, device=DEV)
        cr.convrot_attention(q, k, v, q_offsets=qo, k_offsets=ko, out=out, lse=lse)
        inside = torch.zeros(50, dtype=torch.bool, device=DEV)
        inside[3:40] = True
        assert (out[~inside] == 7).all() and (lse[:, ~inside] == 7).all()
        close(q[3:13], k[:9], v[:9], out[3:13], lse[:, 3:13], 1 / 8, False)
        close(q[13:40], k[9:], v[9:], out[13:40], lse[:, 13:40], 1 / 8, False)


def test_offsets_that_leave_the_tensors_stay_inside():
    """Nothing is read or written out of bounds; sequences that are as they should be
    come out right."""
    rng = np.random.default_rng(5)
    q, k, v = make(rng, [100], [200], 4, 2, 64, torch.bfloat16)
    guard = torch.full((300, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    for qo, ko in (([0, 20, 1 << 30], [0, 50, 1 << 30]), ([0, 20, 10], [0, 50, 40]),
                   ([0, 20, 100], [0, 50, -7]), ([0, 20, -(1 << 31)], [0, 50, 200])):
        for tile in (32, 128):
            out = guard[100:200]
            cr.convrot_attention(q, k, v, tile=tile, out=out,
                                 q_offsets=torch.tensor(qo, dtype=torch.int32, device=DEV),
                                 k_offsets=torch.tensor(ko, dtype=torch.int32, device=DEV))
            torch.cuda.synchronize()
            close(q[:10], k[:50], v[:50], out[:10], None, 1 / 8, False)
            assert (guard[:100] == 7).all() and (guard[200:] == 7).all()


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("n,hq,d,length", [(40, 1, 8, 300000), (70, 1, 64, 220000)])
def test_one_tile_over_so_many_keys_that_the_join_bounds_its_parts(n, hq, d, length, causal):
    rng = np.random.default_rng(n)
    q, k, v = make(rng, [n], [length], hq, 1, d, torch.bfloat16, 4.0)
    out, lse = cr.convrot_attention(q, k, v, causal=causal, return_lse=True)
    close(q, k, v, out, lse, d ** -0.5, causal)


@DTYPES
def test_a_last_round_that_is_split(dtype):
    """More tiles than run at a time: those behind the last whole round go by parts."""
    rng = np.random.default_rng(13)
    n, length, heads, d = 2200, 2100, 33, 128
    q, k, v = make(rng, [n], [length], heads, heads, d, dtype, 3.0)
    for tile in (128, 256):
        assert cr.convrot_attention_workspace_size(q, k, v, tile=tile) > 0
        out, lse = cr.convrot_attention(q, k, v, return_lse=True, tile=tile)
        for h in (0, 15, 30, 31, 32):
            close(q[:, h:h + 1], k[:, h:h + 1], v[:, h:h + 1], out[:, h:h + 1], lse[h:h + 1],
                  d ** -0.5, False)


@pytest.mark.parametrize("n,length,hq,hk,tile", [(2200, 2100, 33, 33, 256), (700, 4000, 2, 2, 128),
                                                 (1, 9000, 8, 2, 0)])
def test_no_workspace(n, length, hq, hk, tile):
    """A call that asks for one does without: no keys are split."""
    rng = np.random.default_rng(14)
    q, k, v = make(rng, [n], [length], hq, hk, 128, torch.bfloat16, 3.0)
    assert cr.convrot_attention_workspace_size(q, k, v, tile=tile) > 0
    none = torch.empty(0, dtype=torch.uint8, device=DEV)
    assert none.data_ptr() == 0
    out, lse = cr.convrot_attention(q, k, v, return_lse=True, tile=tile, workspace=none)
    for h in (0, hq - 1):
        g = h // (hq // hk)
        close(q[:, h:h + 1], k[:, g:g + 1], v[:, g:g + 1], out[:, h:h + 1], lse[h:h + 1],
              128 ** -0.5, False)


@DTYPES
def test_many_sequences(dtype):
    """More than a wave's worth of sequences, some empty."""
    rng = np.random.default_rng(6)
    lens = rng.integers(0, 40, 200).tolist()
    lens[3] = 300
    q, k, v = make(rng, lens, lens, 2, 1, 64, dtype, 2.0)
    for causal in (False, True):
        out, lse = run_packed(q, k, v, lens, lens, causal)
        check_packed(q, k, v, out, lse, lens, lens, causal)


def test_layouts():
    rng = np.random.default_rng(7)
    dt, n, h, d = torch.bfloat16, 150, 4, 64
    mix = dev(rng.standard_normal((2, n, h, 3, d)), dt)
    q, k, v = (mix[:, :, :, i] for i in range(3))
    want = cr.convrot_attention(q.contiguous(), k.contiguous(), v.contiguous())
    assert torch.equal(cr.convrot_attention(q, k, v), want)
    # into columns of a wider tensor that holds the inputs
    wide = torch.cat([t.reshape(2 * n, h * d) for t in (q, k, v)], 1)
    wide = torch.cat([wide, torch.zeros_like(wide[:, :h * d])], 1)
    col = [wide[:, i * h * d:(i + 1) * h * d].view(2, n, h, d) for i in range(4)]
    assert torch.equal(cr.convrot_attention(*col[:3], out=col[3]), want)
    # heads outermost
    hm = [t[0].transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v)]
    assert torch.equal(cr.convrot_attention(*hm), want[0])
    for b in range(2):
        close(q[b], k[b], v[b], want[b], None, 1 / 8, False)


@pytest.mark.parametrize("far", ["tokens", "heads"])
@pytest.mark.parametrize("q,tile", [(1, 0), (40, 128), (300, 256), (300, 0)])
def test_offsets_beyond_32_bits(q, tile, far):
    """Keys, queries and results of which the last lie past 2^32 bytes and 2^31
    elements: the bits of the same call on tensors without gaps."""
    rng = np.random.default_rng(q + tile)
    n, h, d, dt = 1100, 2, 128, torch.bfloat16
    room = torch.empty(n << 21, dtype=dt, device=DEV)
    if far == "tokens":  # column ranges of one wide tensor
        cols = [room.view(n, 1 << 21)[:, i * h * d:(i + 1) * h * d].view(n, h, d)
                for i in range(4)]
    else:  # a head's tokens together
        cols = [torch.as_strided(room, (n, h, d), (d, (n << 21) - 8 * n * d, 1), i * n * d)
                for i in range(4)]
    qc, kc, vc = make(rng, [q], [n], h, h, d, dt)
    for col, x in zip(cols, (qc, kc, vc)):
        col[n - x.shape[0]:] = x
    q_far, out_far = cols[0][n - q:], cols[3][n - q:]
    out_far.fill_(7.0)
    want, want_lse = cr.convrot_attention(qc, kc, vc, causal=True, tile=tile, return_lse=True)
    got, lse = cr.convrot_attention(q_far, cols[1], cols[2], causal=True, tile=tile, out=out_far,
                                    return_lse=True)
    assert torch.equal(got, want) and torch.equal(lse, want_lse)
    close(qc, kc, vc, want, want_lse, 1 / math.sqrt(d), True)


def test_scale_and_large_scores():
    rng = np.random.default_rng(8)
    q, k, v = make(rng, [64], [100], 2, 2, 64, torch.bfloat16)
    for scale in (1e-3, 0.7, 3.0):
        out, lse = cr.convrot_attention(q, k, v, scale=scale, return_lse=True)
        close(q, k, v, out, lse, scale, False)
    # scores of 10^30, all negative, and equal
    big = torch.full_like(q, 1e15)
    out, lse = cr.convrot_attention(big, -big[:1].expand(100, 2, 64), v, return_lse=True)
    want = v.double().mean(0)
    assert ((out.double() - want).abs().max() <= 2.0 ** -7 * v.abs().max()).item()
    assert (lse < -1e28).all().item()


@pytest.mark.parametrize("n,length,hq,hk", [(1, 9000, 8, 2), (3, 700, 4, 4), (100, 3000, 2, 1)])
def test_workspaces(n, length, hq, hk):
    rng = np.random.default_rng(9)
    q, k, v = make(rng, [n], [length], hq, hk, 128, torch.float16, 2.0)
    size = cr.convrot_attention_workspace_size(q, k, v)
    assert size > 0
    want, lse = cr.convrot_attention(q, k, v, return_lse=True)
    close(q, k, v, want, lse, 128 ** -0.5, False)
    guard = torch.full((size + 1024,), 77, dtype=torch.uint8, device=DEV)
    got, got_lse = cr.convrot_attention(q, k, v, workspace=guard[256:256 + size], return_lse=True)
    assert torch.equal(got, want) and torch.equal(got_lse, lse)
    assert torch.equal(cr.convrot_attention(q, k, v), want)
    assert (guard[:256] == 77).all() and (guard[256 + size:] == 77).all()
    for part in (0, 256, size // 2, size - 256):
        got, lse = cr.convrot_attention(q, k, v, workspace=guard[:part], return_lse=True)
        close(q, k, v, got, lse, 128 ** -0.5, False)
        assert (guard[256 + size:] == 77).all()


def test_results_repeat_and_do_not_depend_on_the_device():
    rng = np.random.default_rng(10)
    for n, length, hq, hk, tile in ((300, 900, 4, 2, 0), (1, 5000, 8, 1, 0), (900, 900, 3, 3, 256),
                                    (700, 700, 5, 5, 128)):
        q, k, v = make(rng, [n], [length], hq, hk, 128, torch.bfloat16)
        for causal in (False, True):
            want, lse = cr.convrot_attention(q, k, v, causal=causal, tile=tile, return_lse=True)
            close(q, k, v, want, lse, 128 ** -0.5, causal)
            for cus in (0, 3, 64, 128, 192):
                cr.convrot_set_compute_units(cus)
                try:
                    got = cr.convrot_attention(q, k, v, causal=causal, tile=tile, return_lse=True)
                    assert torch.equal(got[0], want) and torch.equal(got[1], lse)
                finally:
                    cr.convrot_set_compute_units(0)


def test_streams_and_graphs():
    rng = np.random.default_rng(11)
    calls = []
    for n, length, hq, hk in ((200, 300, 4, 2), (2, 6000, 8, 2), (1, 9000, 4, 1)):
        q, k, v = make(rng, [n], [length], hq, hk, 64, torch.bfloat16)
        calls.append((q, k, v, cr.convrot_attention(q, k, v, causal=True)))
    streams = [torch.cuda.Stream() for _ in calls]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(4):
        for s, (q, k, v, _) in zip(streams, calls):
            with torch.cuda.stream(s):
                got.append(cr.convrot_attention(q, k, v, causal=True))
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        assert torch.equal(o, calls[i % 3][3])
    out = [torch.zeros_like(c[3]) for c in calls]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for (q, k, v, _), o in zip(calls, out):
            cr.convrot_attention(q, k, v, causal=True, out=o)
    for _ in range(3):
        for o in out:
            o.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, c[3]) for o, c in zip(out, calls))
        torch.ones(1000, device=DEV).sum().item()
    # other lengths in the same buffers are read at each replay
    used = torch.tensor([9000], dtype=torch.int32, device=DEV)
    q, k, v, _ = calls[2]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cr.convrot_attention(q, k, v, k_lens=used, out=out[2])
    for n in (9000, 1, 4321, 0):
        used.fill_(n)
        graph.replay()
        torch.cuda.synchronize()
        close(q, k[:n], v[:n], out[2], None, 1 / 8, False)


def test_a_block():
    """Projection, norms and rotation in place, attention, output projection: the
    attention half of a block as a model runs it, over two packed sequences."""
    rng = np.random.default_rng(12)
    lens, heads, d = [150, 70], 4, 64
    t, width = sum(lens), heads * d
    x = dev(rng.standard_normal((t, width)), torch.bfloat16)
    w_in = cr.convrot_quantize_mx4(dev(rng.standard_normal((3 * width, width)) * 0.06,
                                       torch.bfloat16), 256)
    w_out = cr.convrot_quantize_mx4(dev(rng.standard_normal((width, width)) * 0.06,
                                        torch.bfloat16), 256)
    weight = dev(1 + 0.1 * rng.standard_normal(d), torch.bfloat16)
    pos = np.stack([np.zeros(t), np.arange(t) // 10, np.arange(t) % 10], 1).astype(np.int64)
    table = cr.convrot_rope_table(dev(pos, torch.int64), (16, 24, 24))
    qkv = cr.convrot_linear_mx4(x, *w_in, 256)
    q, k, v = qkv.view(t, 3, heads, d).unbind(1)
    raw = [f64(y) for y in (q, k, v)]
    q, k = cr.convrot_qk_norm_rope(q, k, table, q_weight=weight, k_weight=weight, q_out=q, k_out=k)
    for y, r in zip((q, k), raw):
        ms = np.sqrt((r ** 2).mean(-1, keepdims=True) + 1e-6)
        want = ref.rotate(r / ms * f64(weight), f64(table), False)
        mag = np.abs(r / ms * f64(weight)).max(-1, keepdims=True)
        assert (np.abs(f64(y) - want) <= 2.0 ** -8 * np.abs(want) + 200 * U * mag).all()
    at = offsets(lens)
    o, lse = cr.convrot_attention(q, k, v, q_offsets=at, k_offsets=at, return_lse=True)
    check_packed(q, k, v, o, lse, lens, lens, False)
    y = cr.convrot_linear_mx4(o.reshape(t, width), *w_out, 256)
    codes, scales = cr.convrot_quantize_mx4(o.reshape(t, width), 256)
    assert torch.equal(y, cr.convrot_gemm_mx4(codes, scales, *w_out))
