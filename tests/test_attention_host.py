"""The rotary table, norm-and-rotation and attention entry points without a GPU:
refusals come before any HIP call, workspace sizes are host arithmetic, and the
oracle's own pins."""

import ctypes
import math
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import int8_gemm_amd as cr
from int8_gemm_amd import attention
from oracle import attention_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(cr.library_path()):
        from int8_gemm_amd import _build
        _build.build()
    return cr.load_library()


# aligned stand-ins, far apart, never dereferenced on these paths
A, B, C, D, E, F = (1 << 32, 1 << 36, 1 << 40, 1 << 42, 1 << 44, 1 << 46)
NAN, INF = float("nan"), float("inf")


def test_table_refusals(lib):
    def st(p=A, kind=1, ts=3, as_=1, tokens=8, dims=(16, 24, 24), theta=1e4, out=B, axes=None):
        arr = (ctypes.c_int32 * max(1, len(dims)))(*dims)
        return lib.convrot_rope_table(p, kind, ts, as_, tokens, len(dims) if axes is None else axes,
                                      arr, theta, 0, out, None)
    assert st(kind=3) == 1 and st(kind=-1) == 1 and st(tokens=-1) == 1
    assert st(axes=0) == 1 and st(dims=(2,) * 9) == 1
    assert st(theta=0.0) == 1 and st(theta=-1.0) == 1 and st(theta=NAN) == 1 and st(theta=INF) == 1
    assert st(dims=(15, 24)) == 3 and st(dims=(0, 24)) == 3 and st(dims=(-2, 24)) == 3
    assert st(dims=(128, 130)) == 3 and st(dims=(258,)) == 3 and st(tokens=(1 << 28) + 1) == 3
    assert st(ts=-1) == 1 and st(as_=-3) == 1 and st(ts=(1 << 40) + 1) == 1
    assert st(p=None) == 1 and st(out=None) == 1
    assert st(p=A + 4) == 4 and st(p=A + 4, kind=0, tokens=0) == 0 and st(out=B + 8) == 4
    assert st(out=A + 176) == 1 and st(p=B + 2040) == 1      # 8 x 3 positions, 8 x 32 x 8 bytes
    assert st(tokens=0, p=None, out=None) == 0


def qk_status(lib, **kw):
    a = attention._QkArgs(q=A, k=B, q_out=C, k_out=D, tokens=10, table=E, table_rows=10,
                          q_heads=4, k_heads=2, d=64, pairs=32, norm=1, eps=1e-6,
                          q_stride=256, q_head_stride=64, k_stride=128, k_head_stride=64,
                          q_out_stride=256, q_out_head_stride=64, k_out_stride=128,
                          k_out_head_stride=64)
    for name, v in kw.items():
        setattr(a, name, v)
    return lib.convrot_qk_norm_rope(ctypes.byref(a), None)


def test_qk_refusals(lib):
    def st(**kw):
        return qk_status(lib, **kw)
    assert lib.convrot_qk_norm_rope(None, None) == 1
    assert st(dtype=2) == 1 and st(norm=3) == 1 and st(norm=-1) == 1
    assert st(eps=-1.0) == 1 and st(eps=NAN) == 1 and st(eps=INF) == 1
    assert st(tokens=-1) == 1 and st(q_heads=0) == 1 and st(k_heads=-1) == 1 and st(d=0) == 1
    assert st(pairs=-4) == 1 and st(d=60, pairs=4) == 3 and st(d=264) == 3
    assert st(q_heads=65537) == 3 and st(pairs=36) == 3 and st(pairs=30) == 3
    assert st(pairs=12, halves=1) == 3 and st(tokens=1 << 31, table_rows=1) == 3
    assert st(row=1, q_heads=513, q_stride=1 << 20, q_out_stride=1 << 20) == 3
    assert st(table_rows=0) == 1 and st(table_rows=3) == 1 and st(table_rows=20) == 1
    assert st(norm=0, q_weight=F) == 1 and st(norm=0, k_weight=F) == 1
    for name in ("q", "k", "q_out", "k_out", "table"):
        assert st(**{name: None}) == 1, name
    for name in ("q", "k", "q_out", "k_out", "table", "q_weight", "k_weight"):
        assert st(**{name: F + 8}) == 4, name
    for name in ("q_stride", "k_stride", "q_out_stride", "k_out_head_stride"):
        assert st(**{name: 260}) == 4 and st(**{name: -256}) == 1
        assert st(**{name: (1 << 40) + 8}) == 1, name
    # outputs onto themselves, each other, inputs, weights and the table
    assert st(q_out_stride=192) == 1 and st(k_out_head_stride=56) == 1
    assert st(k_out=C + 64) == 1 and st(q_out=A + 128) == 1 and st(q_out=B) == 1
    assert st(k_out=A) == 1 and st(q_weight=C + 16) == 1 and st(table=D + 16) == 1
    assert st(q=C, q_stride=512, q_head_stride=128) == 1     # in place, of other strides
    assert st(tokens=0, q=None, k=None, q_out=None, k_out=None, table=None) == 0
    assert st(tokens=0, table_rows=5, k_heads=0, k=None, k_out=None) == 0


def attention_args(**kw):
    a = attention._AttentionArgs(q=A, k=B, v=C, out=D, q_tokens=10, k_tokens=20, batch=1,
                                 q_heads=4, k_heads=2, d=64, scale=0.125, q_stride=256,
                                 q_head_stride=64, k_stride=128, k_head_stride=64, v_stride=128,
                                 v_head_stride=64, out_stride=256, out_head_stride=64)
    for name, v in kw.items():
        setattr(a, name, v)
    return a


def test_attention_refusals(lib):
    def st(ws=None, size=0, **kw):
        return lib.convrot_attention(ctypes.byref(attention_args(**kw)), ws, size, None)
    assert lib.convrot_attention(None, None, 0, None) == 1
    assert st(dtype=5) == 1 and st(q_tokens=-1) == 1 and st(k_tokens=-1) == 1 and st(batch=0) == 1
    assert st(q_heads=0) == 1 and st(k_heads=0) == 1 and st(d=0) == 1 and st(d=-8) == 1
    assert st(k_heads=3) == 3 and st(q_heads=1, k_heads=2) == 3 and st(d=60) == 3 and st(d=264) == 3
    assert st(q_tokens=1 << 30) == 3 and st(k_tokens=(1 << 31) - 1) == 3 and st(batch=1 << 24) == 3
    assert st(batch=3, q_offsets=E) == 1 and st(batch=3, k_offsets=E) == 1
    for scale in (0.0, -0.1, 2.5e38, NAN, INF):
        assert st(scale=scale) == 1
    for tile, d in ((-1, 128), (1, 128), (64, 128), (512, 128), (256, 64), (256, 136)):
        assert st(tile=tile, d=d) == 1
    for name in ("q", "k", "v", "out"):
        assert st(**{name: None}) == 1, name
        assert st(**{name: F + 8}) == 4, name
        for stride in (name + "_stride", name + "_head_stride"):
            assert st(**{stride: 132}) == 4 and st(**{stride: -128}) == 1, stride
    assert st(k_stride=(1 << 22) + 8) == 1 and st(v_stride=(1 << 22) + 8) == 1
    assert st(lse=F + 2) == 4 and st(q_offsets=F + 2) == 4 and st(k_offsets=F + 2) == 4
    assert st(k_lens=F + 1) == 4 and st(ws=F + 128, size=1 << 20) == 4
    # out onto itself, inputs, offsets; lse and the workspace onto anything
    assert st(out_stride=192) == 1 and st(out_head_stride=32) == 1
    assert st(out=A) == 1 and st(out=B + 512) == 1 and st(out=C - 512) == 1
    for name in ("q_offsets", "k_offsets", "k_lens"):
        assert st(**{name: D + 16}) == 1, name
        assert st(lse=E, **{name: E + 156}) == 1, name
        assert st(ws=F, size=4096, **{name: F + 4092}) == 1, name
    for p in (A, B, C, D):
        assert st(lse=p + 64) == 1 and st(ws=p + 256, size=1024) == 1
    assert st(lse=F + 64, ws=F, size=1024) == 1
    assert st(q_tokens=0, q=None, out=None, k=None, v=None) == 0
    assert st(q_tokens=1 << 28, q_heads=64, k_heads=64, batch=1, k_tokens=1, q_stride=4096,
              out_stride=4096, out=1 << 50, q=1 << 55) == 3      # more tiles than a grid holds


def test_column_ranges_do_not_clash(lib):
    """q_out beside k in the columns of one tensor passes every check: the refusal
    that follows is another's."""
    row = 512
    inside = {"q": A, "k": A + 512, "q_out": A, "k_out": A + 512, "q_stride": row,
              "k_stride": row, "q_out_stride": row, "k_out_stride": row}
    assert qk_status(lib, **inside, table=A + 768) == 1            # table inside
    assert qk_status(lib, **{**inside, "k_out": A + 504}) == 4
    assert qk_status(lib, **{**inside, "k_out": A + 496}) == 1     # one chunk into q
    assert qk_status(lib, **{**inside, "k_out": A + 1008}) == 1    # and into the next token's q
    # heads outside of tokens, q_out behind q's tokens of each head
    major = {"q": A, "q_stride": 64, "q_head_stride": 6400, "q_out_stride": 64,
             "q_out_head_stride": 6400, "k": None, "k_out": None, "k_heads": 0}
    assert qk_status(lib, **major, q_out=A + 1280, table=A + 2560) == 1
    assert qk_status(lib, **major, q_out=A + 1264) == 1            # one chunk into q
    assert qk_status(lib, **major, q_out=A + 11536) == 1           # and into the next head's q


def test_workspace_sizes(lib):
    def size(**kw):
        return lib.convrot_attention_workspace_size(ctypes.byref(attention_args(**kw)))
    assert lib.convrot_attention_workspace_size(None) == 0
    assert size(d=60) == 0 and size(batch=0) == 0 and size(scale=0.0) == 0
    # enough tiles for the card, and keys too few to split
    assert size(q_tokens=32760, k_tokens=32760, q_heads=40, k_heads=40, d=128) == 0
    assert size(q_tokens=1, k_tokens=64) == 0
    one = size(q_tokens=1, k_tokens=30000)
    assert one > 0
    cr.convrot_set_compute_units(3)
    try:
        assert size(q_tokens=1, k_tokens=30000) == one
    finally:
        cr.convrot_set_compute_units(0)


@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("d,tile", [(8, 0), (64, 0), (64, 128), (128, 128), (128, 256), (256, 0)])
def test_no_more_parts_than_are_joined(lib, d, tile, causal):
    """The kernel that joins a row's parts holds 512 of their factors. A row of parts takes
    their d + 1 floats each and an entry of 8 bytes."""
    rows = 256 if tile == 256 else 128

    def most(q_tokens, group, k_tokens):
        size = lib.convrot_attention_workspace_size(ctypes.byref(attention_args(
            q_tokens=q_tokens, k_tokens=k_tokens, q_heads=group, k_heads=1, d=d, tile=tile,
            causal=causal)))
        if size == 0:
            return 1
        assert size % rows == 0
        parts, rest = divmod(size // rows - 8, (d + 1) * 4)
        assert rest == 0
        return parts
    counts = [most(q, group, keys) for q, group in ((4, 32), (33, 1), (64, 1), (128, 1))
              for keys in (1 << 14, 1 << 17, 196608, 262144, 300000, 540672, 1 << 20, 1 << 21)]
    assert max(counts) <= 512 and max(counts) > 64


def test_binding_checks_tensors():
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    for call in (lambda: cr.convrot_attention(x, x, x), lambda: cr.convrot_qk_norm_rope(x),
                 lambda: cr.convrot_rope_table(torch.zeros(4, dtype=torch.int64), [8])):
        with pytest.raises(ValueError):          # no device tensors
            call()
    for call in (lambda: cr.convrot_attention(x.float(), x, x),
                 lambda: cr.convrot_qk_norm_rope(x.double()),
                 lambda: cr.convrot_rope_table(torch.zeros(4, dtype=torch.int16), [8])):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        cr.convrot_qk_norm_rope(x, norm="max")
    with pytest.raises(ValueError):
        cr.convrot_qk_norm_rope(x, span="token")

    def heads(t):
        return attention._heads(t, "x", torch.bfloat16, -1)[1:]
    assert heads(x) == (4, 2, 64, 128, 64, 1)
    assert heads(torch.zeros((3, 5, 2, 64), dtype=torch.bfloat16)) == (15, 2, 64, 128, 64, 3)
    wide = torch.zeros((4, 6, 64), dtype=torch.bfloat16)
    assert heads(wide[:, 2:4]) == (4, 2, 64, 384, 64, 1)
    assert heads(wide[:, ::3]) == (4, 2, 64, 384, 192, 1)
    assert heads(wide.transpose(0, 1)) == (6, 4, 64, 64, 384, 1)
    with pytest.raises(ValueError):              # sequences with gaps
        heads(torch.zeros((3, 5, 2, 64), dtype=torch.bfloat16)[:, :4])
    with pytest.raises(ValueError):
        heads(x.transpose(1, 2))
    with pytest.raises(ValueError):
        heads(x[0])
    with pytest.raises(TypeError):
        attention._heads(x.float(), "x", torch.bfloat16, -1)
    with pytest.raises(ValueError):              # another device
        attention._heads(x, "x", torch.bfloat16, 0)


def test_structures_match_the_header_and_it_links_as_c99(lib, tmp_path):
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("no gcc")
    inc = os.path.join(ROOT, "include")
    src = os.path.join(ROOT, "tests", "c", "header_attention_c99.c")
    r = subprocess.run([cc, "-std=c99", "-pedantic", "-Wall", "-Werror", "-fPIC", "-shared", "-I",
                        inc, src, "-o", str(tmp_path / "h.so"), cr.library_path(),
                        "-Wl,--no-undefined", "-Wl,--unresolved-symbols=ignore-in-shared-libs"],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    for struct, name in ((attention._QkArgs, "convrot_qk_args"),
                         (attention._AttentionArgs, "convrot_attention_args")):
        fields = [f for f, _ in struct._fields_]
        c = tmp_path / "o.c"
        c.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"convrot.h\"\n"
                     "int main(void) {"
                     + "".join(f'printf("%zu ", offsetof({name}, {f}));' for f in fields)
                     + f'printf("%zu", sizeof({name})); return 0; }}')
        exe = tmp_path / "o"
        subprocess.run([cc, "-std=c99", "-I", inc, str(c), "-o", str(exe)], check=True)
        got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True,
                                              check=True).stdout.split()]
        assert got == [getattr(struct, f).offset for f in fields] + [ctypes.sizeof(struct)]


def test_packed_arguments():
    for kind, pack in ((attention._QkArgs, attention._pack_qk),
                       (attention._AttentionArgs, attention._pack_attention)):
        values = [0.5 if t is ctypes.c_float else i for i, (_, t) in enumerate(kind._fields_)]
        packed = pack(*values)
        a = kind.from_buffer_copy(packed)
        assert len(packed) == ctypes.sizeof(kind)
        assert [getattr(a, n) or 0 for n, _ in kind._fields_] == values
    names = [n for n, _ in attention._AttentionArgs._fields_]
    assert [names[i] for i in (attention._OUT, attention._LSE, attention._OUT_STRIDE,
                               attention._OUT_HEAD_STRIDE, attention._TOKENS)] == [
        "out", "lse", "out_stride", "out_head_stride", "q_tokens"]


def test_oracle_pins():
    # a quarter turn, and pairs by halves
    v = np.arange(8.0).reshape(1, 1, 8)
    t = np.tile([[[0.0, 1.0]]], (1, 2, 1))
    assert ref.rotate(v, t, False)[0, 0].tolist() == [-1, 0, -3, 2, 4, 5, 6, 7]
    assert ref.rotate(v, t, True)[0, 0].tolist() == [-2, -3, 0, 1, 4, 5, 6, 7]
    a = ref.angles([[2, 3]], (4, 4), 100.0)
    assert np.allclose(a, [[2, 0.2, 3, 0.3]])
    assert np.allclose(ref.angles([[2, 3]], (4, 4), 10000.0, True), [[2, 0.2, 0.03, 0.003]])
    # equal scores average, a mask of the lower right corner, a query that sees nothing
    q, k = np.zeros((3, 2, 8)), np.ones((2, 1, 8))
    v = np.stack([np.full((1, 8), 1.0), np.full((1, 8), 3.0)])
    out, lse, spread = ref.attention(q, k, v, 1.0)
    assert (out == 2).all() and (spread == 2).all() and np.allclose(lse, math.log(2))
    out, lse, _ = ref.attention(q, k, v, 1.0, True)
    assert out[:, 0, 0].tolist() == [0, 1, 2] and lse[0].tolist() == [-np.inf, 0, math.log(2)]
    # query heads read their group's key head
    k2 = np.concatenate([k, 2 * k], 1)
    out, _, _ = ref.attention(q[:, :1].repeat(4, 1), k2, np.concatenate([v, v + 10], 1), 1.0)
    assert out[0, :, 0].tolist() == [2, 2, 12, 12]
