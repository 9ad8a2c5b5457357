"""Host-only checks of the block operators: exported symbols, struct sizes,
argument checks that run before any CUDA call, frequencies, the header as plain
C, and the reference's gradients against differences."""
import ctypes
import math
import os
import re
import shutil
import subprocess

import numpy as np
import pytest

from tests import block_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def bl():
    from communication_compressed_sign_gb300 import build
    build.build()
    from communication_compressed_sign_gb300 import block
    block.load()
    return block


def test_symbols_and_struct_sizes(bl):
    with open(os.path.join(ROOT, "include", "lioncub_block.h")) as f:
        declared = sorted(set(re.findall(r"LIONCUB_API[^;(]*?\b(lioncub_\w+)\s*\(", f.read())))
    assert sorted(bl.EXPORTED) == declared
    lib = ctypes.CDLL(bl.embed.lioncub.LIB_PATH)
    assert all(hasattr(lib, name) for name in declared)
    assert [ctypes.sizeof(t) for t in (bl.PackedRows, bl.Heads, bl.Sequences, bl.ScalingSpec)] == [40, 40, 40, 40]


# Made-up addresses: every call below is refused before anything is launched, or has nothing to do.

def _rows(bl, at, cols, kind=1, stride=None):
    return ctypes.byref(bl.embed.Rows(at, cols if stride is None else stride, kind, 0))


def _packed(bl, at, cols, group=128, kind=0, stride=None, scales=1 << 30, scale_stride=None):
    groups = -(-cols // group) if group > 0 else 1
    return ctypes.byref(bl.PackedRows(at, scales, cols if stride is None else stride,
                                      groups if scale_stride is None else scale_stride, group, kind))


def test_handle_refusals(bl):
    L, arg = bl.load(), bl.embed.lioncub.ERR_ARG
    h = ctypes.c_void_p()
    assert L.lioncub_rms_norm_create(None, 8, 1e-5) == arg
    for dim, eps in ((0, 1e-5), (bl.NORM_MAX_DIM + 1, 1e-5), (8, 0.0), (8, -1.0), (8, float("nan")), (8, float("inf"))):
        assert L.lioncub_rms_norm_create(ctypes.byref(h), dim, eps) == arg and h.value is None
        assert L.lioncub_block_last_error()
    assert L.lioncub_rms_norm_forward(None, 0, *[None] * 9) == arg
    assert L.lioncub_rms_norm_backward(None, 0, *[None] * 11) == arg
    assert L.lioncub_rms_norm_status(None, None, None) == arg
    L.lioncub_rms_norm_destroy(None)
    table = (ctypes.c_double * 512)(*[0.5] * 512)
    assert L.lioncub_rotary_create(None, 8, 8, table, 1.0, 0) == arg
    for head_dim, dim, f, m in ((8, 7, table, 1.0), (8, 10, table, 1.0), (8, 0, table, 1.0), (1, 2, table, 1.0),
                                (bl.ROTARY_MAX_DIM + 2, 8, table, 1.0), (8, 8, None, 1.0), (8, 8, table, float("nan"))):
        assert L.lioncub_rotary_create(ctypes.byref(h), head_dim, dim, f, m, 0) == arg and h.value is None
    for bad in (-0.1, 65536.0, float("nan"), float("inf")):
        table[3] = bad
        assert L.lioncub_rotary_create(ctypes.byref(h), 8, 8, table, 1.0, 0) == arg and h.value is None
    assert L.lioncub_rotary_apply(*[None] * 6, 0, None) == arg
    L.lioncub_rotary_destroy(None)


def test_packing_refusals(bl):
    L, arg, align = bl.load(), bl.embed.lioncub.ERR_ARG, bl.embed.lioncub.ERR_ALIGN
    x, big = 1 << 20, 1 << 40

    def pack(rows, cols, m, p):
        return L.lioncub_pack8(rows, cols, m, p, None)

    for rows, cols in ((-1, 8), (8, -1), (1 << 31, 8), (1, 1 << 39), (1 << 20, 1 << 22)):
        assert pack(rows, cols, _rows(bl, x, abs(cols)), _packed(bl, big, abs(cols))) == arg
    assert pack(8, 8, None, _packed(bl, big, 8)) == arg and pack(8, 8, _rows(bl, x, 8), None) == arg
    assert pack(8, 8, _rows(bl, None, 8), _packed(bl, big, 8)) == arg
    assert pack(8, 8, _rows(bl, x, 8, kind=2), _packed(bl, big, 8)) == arg
    assert pack(8, 8, _rows(bl, x, 8, stride=7), _packed(bl, big, 8)) == arg
    assert pack(8, 8, _rows(bl, x + 2, 8), _packed(bl, big, 8)) == align
    for more in (dict(group=16), dict(group=512), dict(group=-1), dict(kind=2), dict(stride=7), dict(scales=None), dict(scale_stride=0)):
        assert pack(8, 8, _rows(bl, x, 8), _packed(bl, big, 8, **more)) == arg, more
    assert pack(8, 300, _rows(bl, x, 300), _packed(bl, big, 300, scale_stride=2)) == arg
    assert pack(8, 8, _rows(bl, x, 8), _packed(bl, big, 8, scales=(1 << 30) + 2)) == align
    assert pack(8, 8, _rows(bl, x, 8), _packed(bl, x + 16, 8)) == arg and b"overlaps" in L.lioncub_block_last_error()
    assert pack(8, 8, _rows(bl, x, 8), _packed(bl, big, 8, scales=x + 32)) == arg
    assert pack(8, 8, _rows(bl, x, 8), _packed(bl, big, 8, scales=big + 32)) == arg
    wide = bl.NORM_MAX_DIM + 1
    assert pack(1, wide, _rows(bl, x, wide), _packed(bl, big, wide, group=0)) == arg
    assert pack(0, 8, _rows(bl, None, 8), _packed(bl, None, 8)) == 0 and pack(8, 0, _rows(bl, x, 0), _packed(bl, big, 0)) == 0
    assert L.lioncub_unpack8(8, 8, _packed(bl, big, 8), _rows(bl, big, 8), None) == arg
    assert L.lioncub_unpack8(8, 8, None, _rows(bl, big, 8), None) == arg


def test_activation_refusals(bl):
    L, arg = bl.load(), bl.embed.lioncub.ERR_ARG
    r = lambda at, kind=1: _rows(bl, at << 20, 8, kind)  # noqa: E731
    p = lambda at, **more: _packed(bl, at << 20, 8, scales=(at + 1) << 20, **more)  # noqa: E731

    def forward(kind, x, up, out, saved=None, saved_up=None):
        return L.lioncub_activation_forward(8, 8, kind, x, up, out, saved, saved_up, None)

    assert forward(2, r(1), None, r(2)) == arg and forward(-1, r(1), None, r(2)) == arg
    assert forward(0, None, None, r(2)) == arg and forward(0, r(1), None, None) == arg
    assert forward(0, r(1), r(3, 0), r(2)) == arg and forward(0, r(1), None, r(2, 0)) == arg
    assert forward(0, r(1), None, r(2), None, p(4)) == arg
    assert forward(0, r(1), None, r(2), p(4, group=0)) == arg
    assert forward(0, r(1), r(3), r(2), p(4), p(4)) == arg and b"overlaps" in L.lioncub_block_last_error()
    assert forward(0, r(1), None, _rows(bl, (1 << 20) + 32, 8)) == arg

    def backward(dout, x, up, px, pup, dx, dup=None, again=None):
        return L.lioncub_activation_backward(8, 8, 0, dout, x, up, px, pup, dx, dup, again, None)

    assert backward(None, r(2), None, None, None, r(3)) == arg and backward(r(1), r(2), None, None, None, None) == arg
    assert backward(r(1), None, None, None, None, r(3)) == arg and backward(r(1), r(2), None, p(4), None, r(3)) == arg
    assert backward(r(1), r(2), None, None, p(4), r(3)) == arg and backward(r(1), None, r(2), p(4), None, r(3)) == arg
    assert backward(r(1), r(2), None, None, None, r(3), dup=r(6)) == arg
    assert backward(r(1), r(2), r(7), None, None, r(3), dup=r(3)) == arg
    assert backward(r(1), r(2, 0), None, None, None, r(3)) == arg and backward(r(1), r(2), None, None, None, r(3, 0)) == arg


def test_arguments_from_tensors_are_refused(bl):
    """The module that reads arguments from tensors, on tensors that are not the GPU's: nothing reaches the library."""
    torch = pytest.importorskip("torch")
    from communication_compressed_sign_gb300 import Packed, build
    build.build_tensors()
    bl._use_torch()
    t, x = bl._tensors, torch.zeros(4, 64)
    packed = Packed(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 1), 128)
    calls = {
        "pack8": (0, x, packed, 0), "unpack8": (0, packed.codes, packed, x, 0), "activation_forward": (0, 0, x, None, x, None, None, 0),
        "activation_backward": (0, 0, x, x, None, x, None, None, 0),
        "rms_norm_forward": (0, 64, 0, x, None, None, None, None, None, x, 0),
        "rms_norm_backward": (0, 64, 0, x, packed, torch.zeros(4), None, None, x, None, None, None, 0),
        "rotary_apply": (0, 64, 0, x.view(1, 4, 1, 64), x.view(1, 4, 1, 64), None, None, None, 0, 0, 0),
    }
    for name, args in calls.items():
        f = getattr(t, name)
        with pytest.raises(ValueError, match="cuda:0|CUDA device"):
            f(*args)
        with pytest.raises(TypeError, match="arguments"):
            f(*args[:-1])
        with pytest.raises(TypeError, match="arguments"):
            f(*args, 0)
        first = next(i for i, a in enumerate(args) if torch.is_tensor(a))
        for bad in (None, 5, "x", [x]):  # what is not a tensor
            with pytest.raises(ValueError, match="must be a tensor"):
                f(*args[:first], bad, *args[first + 1:])
        with pytest.raises((ValueError, RuntimeError)):
            f(*args[:first], torch.zeros(4, 64).to_sparse(), *args[first + 1:])
    for dim in (63, 0):
        with pytest.raises(ValueError, match="columns"):
            t.rms_norm_forward(0, dim, *calls["rms_norm_forward"][2:])
    with pytest.raises(TypeError):
        t.pack8("0", x, packed, 0)  # no device number
    with pytest.raises(OverflowError):
        t.pack8(1 << 70, x, packed, 0)
    with pytest.raises(ValueError, match="kind"):
        bl._kind("relu")


def test_steps_between_rows(bl):
    """The distance between a view's rows, against what torch's own view of it as a matrix has."""
    torch = pytest.importorskip("torch")
    a, b = torch.zeros(4, 5, 30), torch.zeros(3, 4, 2, 6)
    views = (a[..., :7], a[:, 1:3, :7], a[:, :1, :7], a[:1, :, :7], a[:, ::2, :7], a.transpose(0, 1)[..., :7], a[..., ::2], a[:, :, None, :7],
             a[:1, :1, :7], a[0, :, :9], a[0].t(), a[..., :1], a[:, :, 3:4], a[:, :1].expand(4, 5, 30), b[..., :4], b[:, :, :1, :4],
             b.permute(1, 0, 2, 3)[..., :4], b[:, :, 0], b[:, 1, :, :4], a[0, 0, ::3], a[0, 1:2, :9])
    for t in views:
        cols = t.size(-1)
        n = t.numel() // cols
        if t.is_contiguous():
            continue
        try:
            m = t.view(-1, cols)
            want = "columns" if cols > 1 and m.stride(1) != 1 else m.stride(0) if n > 1 else cols
        except RuntimeError:
            want = "fixed distance"
        if isinstance(want, str):
            with pytest.raises(ValueError, match="columns|fixed distance"):
                bl.embed._step(t, "x", n, cols)
        else:
            assert bl.embed._step(t, "x", n, cols) == want, (t.shape, t.stride())


def test_frequencies(bl):
    f = bl.lioncub_rotary_frequencies(64, 10000.0)
    assert np.allclose(f, 10000.0 ** (-np.arange(32) / 32), rtol=1e-14)
    linear = bl.lioncub_rotary_frequencies(64, 10000.0, bl.ScalingSpec(4.0, 0, 0, 0, bl.SCALING_LINEAR, 0))
    assert np.allclose(linear, np.array(f) / 4, rtol=1e-14)
    base = bl.lioncub_rotary_frequencies(64, 10000.0, bl.ScalingSpec(4.0, 0, 0, 0, bl.SCALING_BASE, 0))
    assert base[0] == 1.0 and math.isclose(base[-1], f[-1] / 4, rel_tol=1e-12)  # the slowest is divided by the factor
    parts = np.array(bl.lioncub_rotary_frequencies(64, 10000.0, bl.ScalingSpec(4.0, 2048.0, 1.0, 32.0, bl.SCALING_PARTS, 0)))
    turns = 2048.0 * np.array(f) / (2 * np.pi)
    assert np.array_equal(parts[turns >= 32], np.array(f)[turns >= 32]) and (turns >= 32).any()
    assert np.allclose(parts[turns <= 1], np.array(f)[turns <= 1] / 4, rtol=1e-14) and (turns <= 1).any()
    assert (np.diff(parts) < 0).all()
    arg = bl.embed.lioncub.ERR_ARG
    out, L = (ctypes.c_double * 512)(), bl.load()
    call = lambda dim, base, s=None, to=out: L.lioncub_rotary_frequencies(dim, base, None if s is None else ctypes.byref(s), to)  # noqa: E731
    assert call(7, 10.0) == arg and call(0, 10.0) == arg and call(bl.ROTARY_MAX_DIM + 2, 10.0) == arg
    assert call(8, 0.5) == arg and call(8, float("nan")) == arg and call(8, 10.0, None, None) == arg
    for s in ((0.5, 0, 0, 0, 1), (float("inf"), 0, 0, 0, 1), (2.0, 0, 0, 0, 4), (2.0, 0, 0, 0, -1), (2.0, 0.0, 1.0, 32.0, 3),
              (2.0, 10.0, 32.0, 32.0, 3), (2.0, 10.0, -1.0, 32.0, 3), (2.0, 10.0, float("nan"), 32.0, 3)):
        assert call(8, 10.0, bl.ScalingSpec(*s, 0)) == arg, s
    assert call(2, 10.0, bl.ScalingSpec(2.0, 0, 0, 0, bl.SCALING_BASE, 0)) == arg


def test_reference_codes():
    table = ref.e4m3_numbers()
    assert table[0x7e] == 448 and table[0x08] == 2.0 ** -6 and table[1] == 2.0 ** -9 and np.isnan(table[0x7f])
    finite = table[:127]
    assert np.array_equal(ref.to_e4m3(finite), np.arange(127)) and np.array_equal(ref.to_e4m3(-finite), np.arange(127) + 128)
    middle = (finite[:-1] + finite[1:]) / 2  # ties go to the even code
    assert np.array_equal(ref.to_e4m3(middle), np.arange(126) + np.arange(126) % 2)
    codes, scales = ref.pack(np.array([[127.0, -63.5, 0.5, 1.5, 0.0]]), "int8", 0)
    assert codes.view(np.int8).tolist() == [[127, -64, 0, 2, 0]] and abs(scales[0, 0] - 1) < 1e-6


def test_reference_gradients_by_differences():
    rng = np.random.default_rng(3)
    x, res, w, dout = rng.normal(size=(3, 11)), rng.normal(size=(3, 11)), rng.normal(size=11), rng.normal(size=(3, 11))
    h, r, _ = ref.norm(x, res, w, 1e-3)
    (dx, _), (dw, _), _ = ref.norm_gradient(dout, h, r, w, None, None)
    step = 1e-6
    for i, j in ((0, 0), (1, 7), (2, 10)):
        e = np.zeros_like(x)
        e[i, j] = step
        diff = ((ref.norm(x + e, res, w, 1e-3)[2] - ref.norm(x - e, res, w, 1e-3)[2]) * dout).sum() / (2 * step)
        assert abs(diff - dx[i, j]) < 1e-8
        diff = ((ref.norm(x, res, w + e[i], 1e-3)[2] - ref.norm(x, res, w - e[i], 1e-3)[2]) * dout).sum() / (2 * step)
        assert abs(diff - dw[j]) < 1e-8
    t = np.linspace(-9, 9, 37)
    for kind in ("silu", "gelu"):
        diff = (ref.value_and_slope(t + step, kind)[0] - ref.value_and_slope(t - step, kind)[0]) / (2 * step)
        assert np.abs(diff - ref.value_and_slope(t, kind)[2]).max() < 1e-8
    # the rotation's transpose, over the squared magnitude, is its inverse
    q, f = rng.normal(size=(4, 2, 10)), [1.0, 0.1, 0.01]
    for inter in (False, True):
        there, _ = ref.rotate(q, [0, 5, -3, 1000], f, 1.5, inter, False)
        back, _ = ref.rotate(there, [0, 5, -3, 1000], f, 1.5, inter, True)
        assert np.allclose(back[..., :6], 2.25 * q[..., :6]) and np.array_equal(back[..., 6:], q[..., 6:])


PROGRAM = r"""
#include "lioncub_block.h"
#include <stdio.h>

int main(void)
{
    lioncub_rms_norm_t n = 0;
    lioncub_rotary_t r = 0;
    double f[4];
    lioncub_rotary_scaling s = {2.0, 0.0, 0.0, 0.0, LIONCUB_SCALING_LINEAR, 0};
    int ok = sizeof(lioncub_packed) == 40 && sizeof(lioncub_heads) == 40 && sizeof(lioncub_sequences) == 40;
    ok = ok && lioncub_rms_norm_create(&n, 0, 1e-5f) == LIONCUB_ERR_ARG && n == 0;
    ok = ok && lioncub_rotary_frequencies(8, 10000.0, &s, f) == LIONCUB_OK && f[0] == 0.5;
    ok = ok && lioncub_rotary_create(&r, 8, 9, f, 1.0f, 0) == LIONCUB_ERR_ARG && r == 0;
    ok = ok && lioncub_block_last_error()[0] != 0;
    printf("%s\n", ok ? "OK" : "FAIL");
    return !ok;
}
"""


def test_header_is_c99_and_links(bl, tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    (tmp_path / "a.c").write_text(PROGRAM)
    libdir = os.path.dirname(bl.embed.lioncub.LIB_PATH)
    r = subprocess.run([cc, "-std=c99", "-pedantic", "-Wall", "-Wextra", "-Werror", f"-I{ROOT}/include",
                        str(tmp_path / "a.c"), f"-L{libdir}", "-llioncub", f"-Wl,-rpath,{libdir}", "-o",
                        str(tmp_path / "a")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(tmp_path / "a")], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "OK", r.stdout + r.stderr
