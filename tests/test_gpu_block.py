"""The block operators on the GPU against their definitions in 64 bits.

Bounds are derived, not fitted; U = 2^-24 is a rounding of fp32.
* Norm: the sum x + residual is rounded once, the squares are added in chains of
  at most 32 and trees and chains of at most 21 more, so rstd is off by at most
  (53 + 6) / 2 U and the result by fewer than 40 U of itself.
* Its gradient: the same for the sum of g * n, which is relative to the sum of
  magnitudes: fewer than 64 U of the magnitude that the reference gives; a
  column's sum of n rows is off by fewer than n + 40 U of its magnitudes.
* Activation: the exponential and the quotient are off by at most 2 units in
  the last place each (4 U), the argument by 6 U: 16 U of the magnitudes, 32 U
  for the derivative.
* Rotary: the angle is off by 2^-27 of a turn, sine and cosine by 4 U more,
  three further roundings: 10 U of |a| + |b|.
A bf16 result must lie between the limits of that range rounded to bf16.
Codes are defined by single roundings and must be equal bit for bit where their
input is exact.
"""
import itertools
import os

import numpy as np
import pytest

from tests import block_reference as ref
from tests.embed_reference import limits

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

T = {"f32": torch.float32, "bf16": torch.bfloat16}
CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
EPS = float(np.float32(1e-5))


@pytest.fixture(scope="module")
def ops():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    import communication_compressed_sign_gb300 as pkg
    return pkg


def _rand(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(T[dtype])


def _strided(x, pad=0, shift=0):
    """The same matrix on the GPU in rows `pad` elements apart, `shift` elements
    into their buffer, the rest poisoned; returns (view, whole buffer)."""
    rows, cols = x.shape
    poison = 77 if x.element_size() == 1 else 777.0
    raw = torch.uint8 if x.element_size() == 1 else x.dtype
    whole = torch.full((rows * (cols + pad) + shift + 16,), poison, dtype=raw, device="cuda")
    view = whole[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    view.copy_(x.view(raw))
    return view.view(x.dtype), whole


def _untouched(whole, rows, cols, pad, shift):
    poison = 77 if whole.element_size() == 1 else 777.0
    rest = whole.clone()
    rest[shift:shift + rows * (cols + pad)].view(rows, -1)[:, :cols] = poison
    assert (rest == poison).all(), "wrote outside its matrix"


def _np(x):
    return x.detach().double().cpu().numpy()


def _bits(x):
    return x.detach().contiguous().view(torch.uint8).cpu().numpy()


def _check(got, exact, magnitude, terms, dtype):
    got = _np(got).reshape(exact.shape)
    low, high = (_np(torch.from_numpy(np.ascontiguousarray(v)).to(dtype)) for v in limits(exact, magnitude, terms))
    bad = ~((low <= got) & (got <= high))
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside their limits, first at {np.argwhere(bad)[:4].tolist()}"


def _packed(ops, rows, cols, code, group, pad=0, shift=0):
    """A Packed to be written in rows apart, with the buffers around it."""
    codes, whole = _strided(torch.zeros(rows, cols, dtype=torch.int8), pad, shift)
    groups = -(-cols // group) if group else 1
    scales, around = _strided(torch.zeros(rows, groups), 3 if pad else 0, 1 if shift else 0)
    return ops.Packed(codes.view(CODES[code]), scales, group), whole, around


def _restored(p, code):
    return ref.unpack(_bits(p.codes).reshape(p.codes.shape), p.scales.cpu().numpy(), code, p.group)


LAYOUTS = [(0, 0), (16, 0), (5, 0), (0, 3), (0, 8)]  # pad, shift


# ---- 8 bits -----------------------------------------------------------------------

@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 7), (3, 8), (5, 77), (2, 264), (33, 192), (9, 771), (4, 2048), (1, 5003)])
@pytest.mark.parametrize("code", list(CODES))
@pytest.mark.parametrize("group", [32, 64, 128, 256, 0])
def test_codes_are_equal_to_the_bit(ops, rows, cols, code, group):
    for kind, (pad, shift) in itertools.product(T, LAYOUTS):
        x = _rand((rows, cols), kind, rows * 7 + cols)
        x[:, ::13] *= 30
        codes, scales = ref.pack(x.float().numpy(), code, group)
        out, whole, around = _packed(ops, rows, cols, code, group, pad, shift)
        xv, _ = _strided(x, pad, shift)
        assert ops.pack8(xv, out=out) is out
        assert np.array_equal(_bits(out.codes).reshape(rows, cols), codes), (kind, pad, shift)
        assert np.array_equal(out.scales.cpu().numpy(), scales), (kind, pad, shift)
        _untouched(whole, rows, cols, pad, shift)
        _untouched(around, rows, scales.shape[1], 3 if pad else 0, 1 if shift else 0)
        back, whole = _strided(torch.zeros(rows, cols, dtype=T[kind]), pad, shift)
        ops.unpack8(out, out=back)
        want = torch.from_numpy(ref.unpack(codes, scales, code, group)).to(T[kind])
        assert torch.equal(back.cpu(), want), (kind, pad, shift)
        _untouched(whole, rows, cols, pad, shift)


@pytest.mark.parametrize("rows,cols,pad", [(7999, 1000, 16), (8200, 1024, 0), (7777, 968, 8), (3900, 2016, 24), (1, 8000008, 0)])
@pytest.mark.parametrize("code,group", [("int8", 32), ("e4m3", 64), ("int8", 256)])
def test_codes_of_many_rows(ops, rows, cols, pad, code, group):
    """Sizes at which a warp takes four chunks at once."""
    x = _rand((rows, cols), "bf16", rows + cols)
    x[0, 3], x[rows - 1, cols - 1] = float("nan"), float("-inf")
    codes, scales = ref.pack(x.float().numpy(), code, group)
    out, whole, around = _packed(ops, rows, cols, code, group, pad)
    ops.pack8(_strided(x, pad, 0)[0], out=out)
    got = _bits(out.codes).reshape(rows, cols)
    assert ((got == codes) | ((got | codes) & 127 == 0)).all()  # a zero may have either sign
    assert np.array_equal(out.scales.cpu().numpy(), scales, equal_nan=True)
    _untouched(whole, rows, cols, pad, 0)
    _untouched(around, rows, scales.shape[1], 3 if pad else 0, 0)
    back, whole = _strided(torch.zeros(rows, cols, dtype=torch.bfloat16), pad, 0)
    ops.unpack8(out, out=back)
    want = torch.from_numpy(ref.unpack(codes, scales, code, group)).to(torch.bfloat16)
    assert torch.equal(back.cpu().nan_to_num(nan=123.0), want.nan_to_num(nan=123.0))
    assert torch.equal(back.cpu().isnan(), want.isnan())
    _untouched(whole, rows, cols, pad, 0)


@pytest.mark.parametrize("cols", [256, 259])
def test_products_are_rounded_before_codes_are(ops, cols):
    """Numbers whose exact product with inv and its fp32 rounding lie on two sides of a border between whole numbers."""
    rng = np.random.default_rng(1)
    a = (1 + rng.random(200000)).astype(np.float32)
    x = (a * (rng.integers(0, 126, a.size) + 0.5) / 127).astype(np.float32)
    inv = (np.float32(127) / a).astype(np.float32)
    rounded, exact = np.rint(x * inv), np.rint(x.astype(np.float64) * inv.astype(np.float64))
    pick = np.flatnonzero(rounded != exact)[:500]
    assert pick.size >= 100
    rows = np.zeros((pick.size, cols), np.float32)
    rows[:, 5] = a[pick]
    rows[:, 6:40] = x[pick][:, None]
    codes, scales = ref.pack(rows, "int8", 128)
    p = ops.pack8(torch.from_numpy(rows).cuda())
    assert np.array_equal(_bits(p.codes).reshape(rows.shape), codes) and np.array_equal(p.scales.cpu().numpy(), scales)
    assert (codes[:, 6].view(np.int8) == rounded[pick]).all()


@pytest.mark.parametrize("code", list(CODES))
@pytest.mark.parametrize("group", [64, 0])
@pytest.mark.parametrize("cols", [256, 77])
def test_codes_of_unusual_groups(ops, code, group, cols):
    x = torch.zeros(12, cols)
    x[1] = -0.0
    x[2, 5] = 1e-35  # below 2^-100: held as zeros
    x[3, 5] = 2.0 ** -100
    x[4, 9], x[5, 9], x[6, 9] = float("inf"), -float("inf"), float("nan")
    x[7] = 3.4e38
    x[8] = torch.linspace(-127, 127, cols)
    x[9] = torch.arange(cols) % 5 * 0.5 - 1
    x[10, 1], x[10, 40] = float("nan"), float("inf")
    x[11] = -1.17e-38
    codes, scales = ref.pack(x.numpy(), code, group)
    p = ops.pack8(x.cuda(), group=group, dtype=CODES[code])
    same = (_bits(p.codes).reshape(12, cols) & 127 == codes & 127) & (codes & 127 == 0) | (_bits(p.codes).reshape(12, cols) == codes)
    assert same.all()  # a zero may have either sign
    assert np.array_equal(p.scales.cpu().numpy(), scales, equal_nan=True)
    y = ops.unpack8(p, out_dtype=torch.float32).cpu()
    whole = slice(0, group) if group else slice(0, cols)
    assert y[4:7, whole].isnan().all() and y[10, whole].isnan().all() and (y[:3] == 0).all() and (y[11] == 0).all()
    if group:
        assert (y[4:7, group:] == 0).all()


def test_packed_rows_and_empty_ones(ops):
    x = _rand((6, 5, 192), "bf16", 1).cuda()
    p = ops.pack8(x)
    assert p.codes.shape == x.shape and p.scales.shape == (6, 5, 2) and p.codes.dtype == torch.int8
    assert torch.equal(ops.unpack8(p), ops.unpack8(ops.pack8(x.view(30, 192))).view(6, 5, 192))
    for shape in ((0, 192), (4, 0), (0,)):
        e = ops.pack8(torch.empty(*shape, device="cuda"))
        assert ops.unpack8(e).shape == shape
    t = x.transpose(0, 1)
    with pytest.raises(ValueError, match="fixed distance"):
        ops.pack8(t)
    halves = ops.Packed(p.codes[..., :128], p.scales[..., :1], 128)  # the columns of whole groups
    assert torch.equal(ops.unpack8(halves), ops.unpack8(p)[..., :128])


# ---- the norm -----------------------------------------------------------------------

DIMS = [(1, 1), (1, 768), (3, 7), (8, 768), (5, 771), (2, 8), (65, 192), (4, 1024), (3, 2048), (2, 2056), (17, 520), (2, 5000), (1, 16384),
        (2, 9001)]


@pytest.mark.parametrize("n,D", DIMS)
@pytest.mark.parametrize("xk,rk", list(itertools.product(T, [None, *T])))
def test_norm(ops, n, D, xk, rk):
    layer = ops.RmsNorm(D, eps=1e-5)
    for (pad, shift), wk, ok in zip(LAYOUTS, (None, "f32", "bf16", "f32", "bf16"), ("bf16", "f32", "bf16", "bf16", "f32")):
        x = _rand((n, D), xk, n + D)
        r = None if rk is None else _rand((n, D), rk, n + D + 1, 3.0)
        w = None if wk is None else 1 + _rand((D,), "f32", D, 0.3).to(T[wk])
        xv, _ = _strided(x, pad, shift)
        rv = None if r is None else _strided(r, pad, shift)[0]
        out, whole = _strided(torch.zeros(n, D, dtype=T[ok]), pad, shift)
        summed, around = _strided(torch.zeros(n, D, dtype=T[ok]), pad, shift)
        saved, codes_around, _ = _packed(ops, n, D, "int8", 128, pad, shift)
        rstd = torch.empty(n, device="cuda")
        layer.forward(xv, None if w is None else w.cuda(), residual=rv, summed=summed, saved=saved, rstd=rstd, out=out)
        h, s, y = ref.norm(_np(x), None if r is None else _np(r), None if w is None else _np(w), EPS)
        _check(out, y, np.abs(y), 40, T[ok])
        _check(rstd, s, s, 40, torch.float32)
        h32 = x.float() if r is None else x.float() + r.float()
        assert torch.equal(summed.cpu(), h32.to(T[ok]))
        codes, scales = ref.pack(h32.numpy(), "int8", 128)
        assert np.array_equal(_bits(saved.codes).reshape(n, D), codes) and np.array_equal(saved.scales.cpu().numpy(), scales)
        for around_it in (whole, around, codes_around):
            _untouched(around_it, n, D, pad, shift)
    assert layer.status() == 0


def _near_codes(p, code, y, err):
    """Each value within half a step of its code's, and scales those of the largest."""
    n, D = y.shape
    width = p.group or D
    scales = np.repeat(p.scales.cpu().numpy().astype(np.float64), width, axis=1)[:, :D]
    top = ref.TOPS[code]
    for g in range(-(-D // width)):
        a = np.abs(y[:, g * width:(g + 1) * width]).max(1)
        assert (np.abs(p.scales.cpu().numpy()[:, g] - a / top) <= a / top * (err + 4) * 2.0 ** -24).all()
    got = _restored(p, code).astype(np.float64)
    # the step around a value: one unit, or 2^-3 of its power of two and at least 2^-9 units
    unit = np.where(scales > 0, np.abs(y) / np.where(scales > 0, scales, 1), 0)
    step = scales if code == "int8" else scales * np.exp2(np.floor(np.log2(np.maximum(unit, 2.0 ** -6))) - 3)
    assert (np.abs(got - y) <= 0.5 * step + np.abs(y) * (err + 8) * 2.0 ** -24 + 1e-30).all()


@pytest.mark.parametrize("n,D", [(1, 1), (5, 192), (9, 771), (3, 2048), (2, 5000), (70, 768)])
@pytest.mark.parametrize("code", list(CODES))
@pytest.mark.parametrize("group", [32, 128, 256, 0])
def test_norm_into_8_bits(ops, n, D, code, group):
    layer = ops.RmsNorm(D, eps=1e-5)
    for pad, shift in LAYOUTS:
        x, r = _rand((n, D), "bf16", 5), _rand((n, D), "bf16", 6)
        w = 1 + _rand((D,), "f32", 7, 0.3)
        out, whole, around = _packed(ops, n, D, code, group, pad, shift)
        saved, _, _ = _packed(ops, n, D, "e4m3", group, pad, shift)
        layer.forward(_strided(x, pad, shift)[0], w.cuda(), residual=_strided(r, pad, shift)[0], out=out, saved=saved)
        h, _, y = ref.norm(_np(x), _np(r), _np(w), EPS)
        _near_codes(out, code, y, 40)
        _untouched(whole, n, D, pad, shift)
        _untouched(around, n, out.scales.shape[1], 3 if pad else 0, 1 if shift else 0)
        codes, scales = ref.pack((x.float() + r.float()).numpy(), "e4m3", group)
        assert np.array_equal(_bits(saved.codes).reshape(n, D), codes) and np.array_equal(saved.scales.cpu().numpy(), scales)


@pytest.mark.parametrize("n,D", DIMS + [(700, 771), (1000, 768)])
@pytest.mark.parametrize("dk,hk,gk", [("bf16", "bf16", "bf16"), ("bf16", "int8", "bf16"), ("f32", "f32", "f32"), ("bf16", "f32", "f32"),
                                      ("f32", "e4m3", "bf16"), ("bf16", "int8", None), ("f32", "bf16", None)])
def test_norm_gradient(ops, n, D, dk, hk, gk):
    layer = ops.RmsNorm(D, eps=1e-5)
    for (pad, shift), wk, ok, group in zip(LAYOUTS, ("f32", None, "bf16", "f32", "bf16"), ("bf16", "f32", "f32", "bf16", "bf16"),
                                           (128, 0, 64, 32, 0)):
        dout, h = _rand((n, D), dk, n * 3 + D), _rand((n, D), "f32" if hk in CODES else hk, D)
        g = None if gk is None else _rand((n, D), gk, D + 2)
        w = None if wk is None else 1 + _rand((D,), "f32", D, 0.3).to(T[wk])
        base = _rand((D,), ok, 9) if pad else None
        rstd = (h.double().square().mean(1) + EPS).rsqrt().float()
        if hk in CODES:
            saved, _, _ = _packed(ops, n, D, hk, group, pad, shift)
            ops.pack8(h.cuda(), out=saved)
            exact_h = _restored(saved, hk).astype(np.float64)
        else:
            saved, exact_h = _strided(h, pad, shift)[0], _np(h)
        dx, whole = _strided(torch.zeros(n, D, dtype=T["f32" if gk is None else gk]), pad, shift)
        again, around = _strided(torch.zeros(n, D, dtype=T[ok]), pad, shift)
        dw = torch.full((D + 2,), 777.0, dtype=T[ok], device="cuda")
        gv = None if g is None else _strided(g, pad, shift)[0]
        layer.backward(_strided(dout, pad, shift)[0], saved, rstd.cuda(), None if w is None else w.cuda(), residual_grad=gv, out=dx,
                       weight_grad=dw[1:-1], weight_base=None if base is None else base.cuda(), again=again)
        (x0, xm), (w0, wm), a0 = ref.norm_gradient(_np(dout), exact_h, _np(rstd), None if w is None else _np(w),
                                                   None if g is None else _np(g), None if base is None else _np(base))
        _check(dx, x0, xm, 64, dx.dtype)
        _check(dw[1:-1], w0, wm, n + 40, T[ok])
        _check(again, a0, np.abs(a0), 4, T[ok])
        assert dw[0] == 777 and dw[-1] == 777
        _untouched(whole, n, D, pad, shift)
        _untouched(around, n, D, pad, shift)
        plain = layer.backward(_strided(dout, pad, shift)[0], saved, rstd.cuda(), None if w is None else w.cuda(), residual_grad=gv,
                               out_dtype=dx.dtype)
        assert torch.equal(plain, dx) or D % 8 == 0  # without a weight gradient; a new matrix may allow wider moves
    assert layer.status() == 0


@pytest.mark.parametrize("n,D", [(30000, 768), (30000, 771), (12000, 2048), (40000, 192), (2000, 8200), (700, 16384), (600, 16383), (5000, 520)])
@pytest.mark.parametrize("hk", ["f32", "int8"])
def test_norm_gradient_of_many_rows(ops, n, D, hk):
    """Rows enough that every place of the rings is used several times."""
    g = torch.Generator(device="cuda").manual_seed(n + D)
    rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    dout, res = rand(n, D).bfloat16(), rand(n, D)
    h, w = rand(n, D), 1 + 0.1 * rand(D)
    rstd = (h.double().square().mean(1) + EPS).rsqrt().float()
    saved = h if hk == "f32" else ops.pack8(h, group=64)
    h = h if hk == "f32" else ops.unpack8(saved, out_dtype=torch.float32)
    layer = ops.RmsNorm(D)
    dw, again = torch.empty(D, device="cuda"), torch.empty(n, D, dtype=torch.bfloat16, device="cuda")
    dx = layer.backward(dout, saved, rstd, w, residual_grad=res, weight_grad=dw, again=again, out_dtype=torch.float32)
    worst = 0.0
    dw0, wm = torch.zeros(D, dtype=torch.float64, device="cuda"), torch.zeros(D, dtype=torch.float64, device="cuda")
    for part in torch.arange(n, device="cuda").split(4096):
        d, hh, r = dout[part].double(), h[part].double(), rstd[part].double()[:, None]
        nn, gg = hh * r, d * w.double()
        exact = r * (gg - nn * (gg * nn).mean(1, keepdim=True)) + res[part].double()
        mag = r * (gg.abs() + nn.abs() * (gg * nn).abs().mean(1, keepdim=True)) + res[part].double().abs()
        worst = max(worst, ((dx[part].double() - exact).abs() / mag).max().item())
        y = nn * w.double()
        assert ((again[part].double() - y).abs() <= y.abs() * (2.0 ** -8 + 2.0 ** -20)).all()
        dw0 += (d * nn).sum(0)
        wm += (d * nn).abs().sum(0)
    assert worst < 64 * 2.0 ** -24
    # a column's chain: one row of each ring's turn, then the teams and blocks
    assert ((dw.double() - dw0).abs() <= wm * (n / 152 + 200) * 2.0 ** -24).all()
    assert torch.equal(dx, layer.backward(dout, saved, rstd, w, residual_grad=res, weight_grad=dw, out_dtype=torch.float32))
    assert layer.status() == 0


def test_norm_gradient_of_no_rows_and_in_place(ops):
    D = 264
    layer = ops.RmsNorm(D)
    dw, base = torch.full((D,), 5.0, device="cuda"), _rand((D,), "f32", 1).cuda()
    none, no_rstd = torch.empty(0, D, device="cuda"), torch.empty(0, device="cuda")
    assert layer.forward(none, rstd=no_rstd).shape == (0, D)
    layer.backward(none, none, no_rstd, weight_grad=dw)
    assert (dw == 0).all()
    layer.backward(none, none, no_rstd, weight_grad=dw, weight_base=base)
    assert torch.equal(dw, base)
    for n in (1, 37):
        x, r, dout = (_rand((n, D), "f32", k).cuda() for k in range(3))
        rstd = torch.empty(n, device="cuda")
        summed = torch.empty_like(x)
        y = layer.forward(x, base, residual=r, summed=summed, rstd=rstd)
        xs, rs = x.clone(), r.clone()
        assert torch.equal(layer.forward(xs, base, residual=rs, summed=rs, out=xs), y) and torch.equal(rs, summed) and torch.equal(xs, y)
        dx = layer.backward(dout, summed, rstd, base, residual_grad=r, weight_grad=dw)
        more = base.clone()
        ds, hs, gs = dout.clone(), summed.clone(), r.clone()
        assert torch.equal(layer.backward(ds, hs, rstd, base, residual_grad=gs, out=gs, again=hs, weight_grad=more, weight_base=more), dx)
        assert torch.equal(gs, dx) and torch.equal(more, dw + base) and torch.equal(ds, dout)
        assert torch.equal(hs, layer.forward(summed, base)) or (hs - layer.forward(summed, base)).abs().max() < 1e-5
        assert torch.equal(layer.backward(ds, summed, rstd, base, residual_grad=r, out=ds), dx) and torch.equal(ds, dx)


def test_norm_of_unusual_rows(ops):
    """Rows of zeros, of one value that outweighs the rest, and with an infinity or a NaN: each by itself."""
    for D in (768, 771):
        x = _rand((6, D), "f32", D)
        x[0] = 0
        x[1, 3] = 1e15
        x[2, 5], x[3, 5] = float("inf"), float("nan")
        x[4] = 1e-20
        layer = ops.RmsNorm(D, eps=1e-5)
        y = layer.forward(x.cuda()).cpu()
        assert (y[0] == 0).all() and y[3].isnan().all() and y[2, 5].isnan() and (y[2, :5] == 0).all()
        _, _, want = ref.norm(_np(x[[1, 4, 5]]), None, None, EPS)
        _check(y[[1, 4, 5]], want, np.abs(want), 40, torch.float32)


# ---- the activation ----------------------------------------------------------------------

@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 8), (5, 77), (33, 192), (9, 771), (4, 2048), (1, 5003)])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("xk", list(T))
def test_activation(ops, rows, cols, kind, gated, xk):
    dtype = T[xk]
    for (pad, shift), (code, group) in zip(LAYOUTS, ((None, 0), ("int8", 128), ("e4m3", 32), ("int8", 256), ("e4m3", 64))):
        x, up, dout = (_rand((rows, cols), xk, rows + 5 * k, 3.0) for k in range(3))
        xv, uv, dv = (_strided(v, pad, shift)[0] for v in (x, up, dout))
        uv = uv if gated else None
        bufs = [_strided(torch.zeros(rows, cols, dtype=dtype), pad, shift) for _ in range(4)]
        out, dx, dup, again = (b[0] for b in bufs)
        saved = saved_up = None
        if code:
            saved = _packed(ops, rows, cols, code, group, pad, shift)[0]
            saved_up = _packed(ops, rows, cols, code, group, pad, shift)[0] if gated else None
        ops.activation(xv, uv, kind=kind, out=out, saved=saved, saved_up=saved_up)
        x64, u64, d64 = _np(x), _np(up) if gated else 1.0, _np(dout)
        f, fm, slope, sm = ref.value_and_slope(x64, kind)
        _check(out, f * u64, fm * np.abs(u64), 16, dtype)
        if code:
            codes, scales = ref.pack(x.float().numpy(), code, group)
            assert np.array_equal(_bits(saved.codes).reshape(rows, cols), codes) and np.array_equal(saved.scales.cpu().numpy(), scales)
            x64 = _restored(saved, code).astype(np.float64)
            u64 = _restored(saved_up, code).astype(np.float64) if gated else 1.0
            f, fm, slope, sm = ref.value_and_slope(x64, kind)
        ops.activation_backward(dv, saved or xv, (saved_up or uv) if gated else None, kind=kind, dx=dx, dup=dup if gated else None,
                                again=again)
        _check(dx, d64 * u64 * slope, np.abs(d64 * u64) * sm, 32, dtype)
        _check(again, f * u64, fm * np.abs(u64), 16, dtype)
        if gated:
            _check(dup, d64 * f, np.abs(d64) * fm, 16, dtype)
        for _, whole in bufs[:2] + bufs[3:] + (bufs[2:3] if gated else []):
            _untouched(whole, rows, cols, pad, shift)


@pytest.mark.parametrize("rows,cols", [(3, 1000), (40, 256), (1, 8), (9, 264), (2, 96), (4, 77)])
@pytest.mark.parametrize("kinds", [("int8", 32, "e4m3", 256), ("e4m3", 128, "int8", 64), ("int8", 256, "int8", 32)])
@pytest.mark.parametrize("xk", list(T))
def test_two_saved_matrices_of_different_codes(ops, rows, cols, kinds, xk):
    """Codes, groups and what is not finite of one are no matter of the other's."""
    code, group, code_up, group_up = kinds
    x, up = (_rand((rows, cols), xk, rows + k, 3.0) for k in range(2))
    x[0, 0], x[-1, cols // 2] = float("nan"), float("inf")
    up[0, cols - 1], up[rows // 2, cols // 3] = float("-inf"), 1e-35
    saved, *rest = _packed(ops, rows, cols, code, group, 16)
    saved_up, *rest_up = _packed(ops, rows, cols, code_up, group_up, 16)
    ops.activation(x.cuda(), up.cuda(), kind="silu", saved=saved, saved_up=saved_up)
    for p, v, c, g, (whole, around) in ((saved, x, code, group, rest), (saved_up, up, code_up, group_up, rest_up)):
        codes, scales = ref.pack(v.float().numpy(), c, g)
        got = _bits(p.codes).reshape(rows, cols)
        assert ((got == codes) | ((got | codes) & 127 == 0)).all()  # a zero may have either sign
        assert np.array_equal(p.scales.cpu().numpy(), scales, equal_nan=True)
        _untouched(whole, rows, cols, 16, 0)
        _untouched(around, rows, scales.shape[1], 3, 0)
        only = ops.pack8(v.cuda(), group=g, dtype=CODES[c])
        assert np.array_equal(_bits(only.codes), _bits(p.codes))


@pytest.mark.parametrize("pad,shift", [(4, 0), (0, 4), (4, 4), (12, 8)])
def test_fp32_rows_between_two_alignments(ops, pad, shift):
    """Rows that begin at multiples of 16 bytes, only some of them of 32: results are those of rows in one piece."""
    rows, cols = 37, 192
    plain = [_rand((rows, cols), "f32", k, 3.0).cuda() for k in range(3)]
    weight = _rand((cols,), "f32", 9).cuda()

    def run(pad, shift):
        x, up, dout = (_strided(v.cpu(), pad, shift)[0] for v in plain)
        w = _strided(weight.cpu()[None], pad, shift)[0][0]
        made = []

        def new():
            made.append(_strided(torch.zeros(rows, cols), pad, shift))
            return made[-1][0]

        p, q = (_packed(ops, rows, cols, "int8", 32, 16)[0] for _ in range(2))
        ops.pack8(x, out=p)
        ops.unpack8(p, out=new())
        ops.activation(x, up, kind="silu", out=new(), saved=q)
        ops.activation_backward(dout, x, up, kind="gelu", dx=new(), dup=new(), again=new())
        layer = ops.RmsNorm(cols)
        rstd = torch.empty(rows, device="cuda")
        summed = new()
        layer.forward(x, w, residual=up, summed=summed, rstd=rstd, out=new())
        grad = torch.empty(cols + 4, device="cuda")[shift and 4:][:cols]
        layer.backward(dout, summed, rstd, w, residual_grad=up, out=new(), weight_grad=grad, again=new())
        for _, whole in made:
            _untouched(whole, rows, cols, pad, shift)
        return [v.cpu().clone() for v, _ in made] + [rstd.cpu(), grad.cpu(), p.scales.cpu(), p.codes.cpu(), q.scales.cpu(), q.codes.cpu()]

    for k, (a, b) in enumerate(zip(run(0, 0), run(pad, shift))):
        assert torch.equal(a, b), k


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_activation_far_out(ops, kind):
    x = torch.tensor([0.0, -0.0, 1e-30, 20.0, -20.0, 80.0, -80.0, 90.0, -90.0, 1e10, -1e10, 1e19, -1e19, 3e38, -3e38], device="cuda")
    f, fm, slope, sm = ref.value_and_slope(_np(x).clip(-1e5, 1e5), kind)
    f = np.where(np.abs(_np(x)) > 1e5, np.maximum(_np(x), 0), f)
    y = ops.activation(x.view(1, -1), kind=kind)
    _check(y, f.reshape(1, -1), np.abs(fm).reshape(1, -1) + np.abs(f).reshape(1, -1), 16, torch.float32)
    dx = ops.activation_backward(torch.ones_like(x).view(1, -1), x.view(1, -1), kind=kind)
    assert dx.isfinite().all()
    assert (dx.cpu()[0] - torch.from_numpy(np.where(_np(x) > 20, 1.0, np.where(_np(x) < -20, 0.0, slope)))).abs().max() < 2e-5
    bad = torch.tensor([[float("nan")] * 8], device="cuda")
    assert ops.activation(bad, kind=kind).isnan().all() and ops.activation_backward(bad, x[:8].view(1, 8), kind=kind).isnan().all()


def test_activation_in_place_and_side_by_side(ops):
    both = _rand((19, 2 * 96), "bf16", 3).cuda()
    x, up = both[:, :96], both[:, 96:]
    dout = _rand((19, 96), "bf16", 4).cuda()
    y = ops.activation(x, up, kind="silu")
    dx, dup = ops.activation_backward(dout, x, up, kind="silu")
    z = both.clone()
    assert torch.equal(ops.activation(z[:, :96], z[:, 96:], kind="silu", out=z[:, :96]), y) and torch.equal(z[:, 96:], up)
    z = both.clone()
    ops.activation_backward(dout, z[:, :96], z[:, 96:], kind="silu", dx=z[:, :96], dup=z[:, 96:])
    assert torch.equal(z[:, :96], dx) and torch.equal(z[:, 96:], dup)
    assert ops.activation(torch.empty(0, 5, device="cuda")).shape == (0, 5)


@pytest.mark.parametrize("rows,cols", [(300, 128), (70, 40), (13, 640), (1, 64), (129, 8), (5, 1032)])
@pytest.mark.parametrize("code,group", [("int8", 32), ("e4m3", 128), ("int8", 256)])
def test_rows_narrower_than_a_warps_chunks(ops, rows, cols, code, group):
    """Rows out of wider ones, whole groups of columns or not, of several a warp: each as by itself in one piece."""
    wide = _rand((rows, 3 * cols + 8), "bf16", rows + cols).cuda()
    x, up, dout = wide[:, :cols], wide[:, cols:2 * cols], wide[:, 2 * cols:3 * cols]
    apart = [ops.Packed.empty((rows, cols + 256), group=group, dtype=CODES[code]) for _ in range(2)]
    groups = -(-cols // group)
    saved, saved_up = (ops.Packed(p.codes[:, :cols], p.scales[:, :groups], group) for p in apart)
    y = ops.activation(x, up, kind="silu", saved=saved, saved_up=saved_up)
    f, fm, _, _ = ref.value_and_slope(_np(x), "silu")
    _check(y, f * _np(up), fm * np.abs(_np(up)), 16, torch.bfloat16)
    for p, m in ((saved, x), (saved_up, up)):
        codes, scales = ref.pack(m.float().cpu().numpy(), code, group)
        assert np.array_equal(_bits(p.codes).reshape(rows, cols), codes) and np.array_equal(p.scales.cpu().numpy(), scales)
        assert torch.equal(ops.unpack8(p, out_dtype=torch.float32).cpu(), torch.from_numpy(ref.unpack(codes, scales, code, group)))
        q = ops.pack8(m, group=group, dtype=CODES[code])
        assert np.array_equal(_bits(q.codes).reshape(rows, cols), codes) and np.array_equal(q.scales.cpu().numpy(), scales)
    again = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    dx, dup = ops.activation_backward(dout, saved, saved_up, kind="silu", again=again)
    x64, u64, d64 = _restored(saved, code).astype(np.float64), _restored(saved_up, code).astype(np.float64), _np(dout)
    f, fm, slope, sm = ref.value_and_slope(x64, "silu")
    _check(dx, d64 * u64 * slope, np.abs(d64 * u64) * sm, 32, torch.bfloat16)
    _check(dup, d64 * f, np.abs(d64) * fm, 16, torch.bfloat16)
    _check(again, f * u64, fm * np.abs(u64), 16, torch.bfloat16)


# ---- rotary positions ----------------------------------------------------------------------

def _frequencies(dim, base=10000.0):
    return base ** (-2.0 * np.arange(dim // 2) / dim)


@pytest.mark.parametrize("B,S,H,K,D,R", [(1, 1, 1, 1, 2, 2), (2, 3, 2, 1, 64, 64), (1, 17, 12, 12, 64, 32), (3, 5, 7, 3, 80, 40),
                                         (2, 4, 32, 8, 128, 128), (1, 2, 3, 0, 256, 64), (2, 3, 5, 2, 66, 22), (1, 3, 2, 2, 96, 48),
                                         (4, 1, 1, 0, 24, 8), (3, 7, 4, 8, 80, 20), (1, 40, 3, 2, 1024, 1024)])
@pytest.mark.parametrize("kind", list(T))
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary(ops, B, S, H, K, D, R, kind, interleaved):
    rot = ops.Rotary(D, rotary_dim=R, interleaved=interleaved, magnitude=1.25)
    whole = _rand((B, S, H + 2 * K + 1, D), kind, B * S + H)
    whole_t = _rand((B, H + K, S, D), kind, B + S)
    for where, shift in itertools.product(("own", "fused", "transposed"), (0, 1)):
        def on_gpu(t):
            buf = torch.empty(t.numel() + 8, dtype=t.dtype, device="cuda")[shift:shift + t.numel()].view(t.shape)
            return buf.copy_(t)
        if where == "own":
            q, k = on_gpu(whole[:, :, :H].contiguous()), on_gpu(whole[:, :, H:H + K].contiguous())
        elif where == "fused":
            buf = on_gpu(whole)
            q, k = buf[:, :, :H], buf[:, :, H:H + K]
        else:
            buf = on_gpu(whole_t)
            q, k = buf[:, :H].transpose(1, 2), buf[:, H:].transpose(1, 2)
        for positions, first in ((None, 0), (None, 12345), ("i32", 0), ("i64", 0)):
            if positions is None:
                at, p = np.tile(np.arange(S) + first, B), None
            else:
                at = np.random.default_rng(S).integers(-1000, 1 << 20, B * S)
                p = torch.from_numpy(at).to(torch.int32 if positions == "i32" else torch.int64).view(B, S).cuda()
            for inverse in (False, True):
                go = rot.backward if inverse else rot.forward
                got = go(q, k if K else None, positions=p, first_position=first)
                got = got if K else (got,)
                for x, y in zip((q, k), got):
                    exact, mag = ref.rotate(_np(x).reshape(B * S, -1, D), at, _frequencies(R), 1.25, interleaved, inverse)
                    _check(y, exact, mag, 10, T[kind])
                    assert torch.equal(y[..., R:], x[..., R:])
        # in place, also side by side in one buffer
        want = rot.forward(q, k if K else None, first_position=7)
        want = want if K else (want,)
        rest = None if where != "fused" else buf[:, :, H + K:].clone()
        rot.forward(q, k if K else None, first_position=7, q_out=q, k_out=k if K else None)
        assert torch.equal(q, want[0]) and (not K or torch.equal(k, want[1]))
        assert rest is None or torch.equal(buf[:, :, H + K:], rest)


@pytest.mark.parametrize("B,S,H,K,D,R", [(3, 1777, 2, 1, 80, 20), (2, 3001, 1, 2, 80, 40), (1, 1217, 3, 0, 64, 64), (7, 701, 2, 2, 20, 10),
                                         (1, 5003, 1, 1, 66, 22), (5, 433, 4, 3, 128, 96), (4, 999, 2, 1, 24, 8)])
@pytest.mark.parametrize("kind", list(T))
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_of_many_places(ops, B, S, H, K, D, R, kind, interleaved):
    """Several places a block, of two sequences too, and a last block with fewer."""
    rot = ops.Rotary(D, rotary_dim=R, interleaved=interleaved)
    buf = _rand((B, S, H + K + 1, D), kind, B * S + H).cuda()
    at = np.random.default_rng(S).integers(0, 1 << 20, B * S)
    p = torch.from_numpy(at).view(B, S).cuda()
    q, k = buf[:, :, :H], buf[:, :, H:H + K]
    outs = [torch.full((B, S, h, D + 8), 777.0, dtype=T[kind], device="cuda") for h in (H, K)]
    to = [o[..., :D] for o in outs]
    rot.forward(q, k if K else None, positions=p, q_out=to[0], k_out=to[1] if K else None)
    for x, y, o in zip((q, k), to, outs):
        if x.shape[2]:
            exact, mag = ref.rotate(_np(x).reshape(B * S, -1, D), at, _frequencies(R), 1.0, interleaved, False)
            _check(y, exact, mag, 10, T[kind])
            assert torch.equal(y[..., R:], x[..., R:])
            assert (o[..., D:] == 777.0).all()
    rest = buf[:, :, H + K:].clone()
    rot.forward(q, k if K else None, positions=p, q_out=q, k_out=k if K else None)
    assert torch.equal(q, to[0]) and torch.equal(k, to[1]) and torch.equal(buf[:, :, H + K:], rest)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_of_fp32_heads_between_two_alignments(ops, interleaved):
    """Heads that begin at multiples of 16 bytes but not of 32: results are those of others."""
    rot = ops.Rotary(96, rotary_dim=64, interleaved=interleaved)
    q = _rand((3, 50, 4, 96), "f32", 5).cuda()
    want = rot.forward(q, first_position=9)
    for shift, pad in ((4, 0), (0, 4), (4, 4), (12, 12)):
        x, y = (torch.full((q.numel() // 96 * (96 + pad) + shift,), 777.0, device="cuda") for _ in range(2))
        xv, yv = (t[shift:].view(3, 50, 4, 96 + pad)[..., :96] for t in (x, y))
        xv.copy_(q)
        rot.forward(xv, first_position=9, q_out=yv)
        assert torch.equal(yv, want) and torch.equal(xv, q)
        assert (y[:shift] == 777.0).all() and (y[shift:].view(3, 50, 4, 96 + pad)[..., 96:] == 777.0).all()


def test_rotary_scalings_far_positions_and_adjoint(ops):
    D = 128
    turns = _frequencies(D)
    x = _rand((1, 5, 3, D), "f32", 8)
    at = np.array([0, 1 << 20, -(1 << 20), (1 << 30) + 1, 99_999_999])
    p = torch.from_numpy(at).view(1, 5).cuda()
    for scaling in (None, ops.RotaryScaling("linear", 4.0), ops.RotaryScaling("base", 4.0), ops.RotaryScaling("parts", 4.0, length=2048),
                    ops.RotaryScaling("parts", 8.0, length=8192, low=1.0, high=4.0, magnitude=1.0)):
        rot = ops.Rotary(D, scaling=scaling)
        f, m = np.array(rot.frequencies), rot.magnitude
        if scaling is None:
            assert np.allclose(f, turns, rtol=1e-14) and m == 1
        elif scaling.kind == "parts" and scaling.magnitude is None:
            assert abs(m - (0.1 * np.log(4.0) + 1)) < 1e-12
        exact, mag = ref.rotate(_np(x[0]), at, f, float(np.float32(m)), False, False)
        # beside 10 U: position * 2^-52 turns * frequency here and as much in the reference's own product
        extra = np.abs(at)[:, None, None] * (2 * 2 * np.pi * 2.0 ** -52) / 2.0 ** -24
        _check(rot.forward(x.cuda(), positions=p), exact, mag * (10 + extra), 1, torch.float32)
    rot = ops.Rotary(D, rotary_dim=64)
    y = _rand((1, 5, 3, D), "f32", 9)
    forward, backward = _np(rot.forward(x.cuda(), positions=p)), _np(rot.backward(y.cuda(), positions=p))
    assert abs((forward * _np(y)).sum() - (_np(x) * backward).sum()) < 5 * 3 * D * 10 * 2.0 ** -24 * 16
    given = ops.Rotary(4, frequencies=[0.0, 1.5707963267948966])
    one = given.forward(torch.tensor([[[1.0, 2.0, 0.0, 0.0]]], device="cuda").view(1, 1, 1, 4), first_position=2)
    assert torch.allclose(one.view(-1).cpu(), torch.tensor([1.0, -2.0, 0.0, 0.0]), atol=1e-6)  # half a turn of pair (1, 3)


def test_rotary_of_broadcast_inputs_and_nothing(ops):
    rot = ops.Rotary(64)
    one = _rand((1, 7, 1, 64), "bf16", 2).cuda()
    many = one.expand(3, 7, 4, 64)
    y = rot.forward(many)
    assert torch.equal(y, rot.forward(many.contiguous())) and y.shape == (3, 7, 4, 64)
    assert torch.equal(rot.forward(one[0]), rot.forward(one)[0])  # without a batch dimension
    for shape in ((0, 7, 2, 64), (2, 0, 2, 64), (2, 7, 0, 64)):
        assert rot.forward(torch.empty(shape, device="cuda")).shape == shape


# ---- refusals that need tensors ---------------------------------------------------------------

def test_refusals(ops):
    E = ops.LionCubError
    x, w = _rand((4, 64), "f32", 1).cuda(), torch.ones(64, device="cuda")
    layer = ops.RmsNorm(64)
    rstd = torch.empty(4, device="cuda")
    for bad in (x.half(), x.cpu(), x.double(), x[:, :32], x.t()):
        with pytest.raises(ValueError):
            layer.forward(bad)
    with pytest.raises(ValueError, match="gradient"):
        layer.forward(x, w.clone().requires_grad_())
    for kw in (dict(residual=x[:3]), dict(summed=x.half()), dict(rstd=rstd[:3]), dict(rstd=rstd.double()), dict(out=x[:, :32]),
               dict(saved=ops.Packed.empty((4, 32))), dict(saved=ops.Packed(x.to(torch.uint8), rstd.view(4, 1)))):
        with pytest.raises(ValueError):
            layer.forward(x, w, **kw)
    buf = torch.zeros(5 * 64, device="cuda")
    for kw in (dict(out=buf[32:288].view(4, 64)), dict(summed=buf[64:].view(4, 64)), dict(out=x, summed=x),
               dict(rstd=buf[:4]), dict(residual=buf[64:].view(4, 64), summed=buf[:256].view(4, 64))):
        with pytest.raises(E, match="overlaps"):
            layer.forward(buf[:256].view(4, 64), w, **{**dict(out=torch.empty_like(x)), **kw} if "out" not in kw else kw)
    for kw in (dict(weight_base=w), dict(weight_grad=x[0].contiguous(), weight_base=w.bfloat16())):
        with pytest.raises(E):
            layer.backward(x, x.clone(), rstd, w, **kw)
    with pytest.raises(E, match="overlaps"):
        layer.backward(x, buf[:256].view(4, 64), rstd, w, weight_grad=buf[100:164])
    with pytest.raises(ValueError):
        ops.activation(x, kind="relu")
    with pytest.raises(E):
        ops.activation(x, out=torch.empty_like(x), saved=ops.Packed.empty((4, 64), group=0))
    with pytest.raises(E):
        ops.pack8(x, group=48)
    rot = ops.Rotary(64)
    q = _rand((2, 4, 3, 64), "f32", 1).cuda()
    for bad in (q.half(), q[..., :32], q[0, 0], q.cpu()):
        with pytest.raises(ValueError):
            rot.forward(bad)
    with pytest.raises(ValueError):
        rot.forward(q, positions=torch.zeros(2, 3, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        rot.forward(q, positions=torch.zeros(2, 4, device="cuda"))
    with pytest.raises(ValueError):
        rot.forward(q, k_out=q)
    with pytest.raises(E, match="type"):
        rot.forward(q, q.bfloat16())
    with pytest.raises(E, match="share memory"):
        rot.forward(q, q_out=q[:, :, :1].expand(2, 4, 3, 64))
    fused = torch.zeros(2, 4, 8, 64, device="cuda")
    for a, b in ((fused[:, :, 1:4], fused[:, :, :3]), (fused[:, :3].view(2, 3, 8, 64)[:, :, :3], fused[:, 1:, :3])):
        with pytest.raises(E, match="overlap"):
            rot.forward(a, q_out=b)
    with pytest.raises(E, match="overlap"):
        rot.forward(fused[:, :, :3], fused[:, :, 3:6], q_out=fused[:, :, :3], k_out=fused[:, :, 2:5])
    rot.forward(fused[:, :, :3], q_out=fused[:, :, 3:6])  # other heads of one buffer
    rot.forward(fused[:, :, :3], fused[:, :, 7:], q_out=fused[:, :, 3:6], k_out=fused[:, :, 6:7])
    flat = fused.transpose(1, 2).contiguous().transpose(1, 2)  # heads outside places
    rot.forward(flat[:, :, :3], flat[:, :, 7:], q_out=flat[:, :, :3], k_out=flat[:, :, 6:7])
    with pytest.raises(E):
        rot.forward(q, first_position=1 << 41)
    for closed in (layer, rot):
        closed.close()
        closed.close()
    with pytest.raises(E, match="closed"):
        layer.forward(x)
    with pytest.raises(E, match="closed"):
        rot.forward(q)


# ---- streams, graphs, sizes, faults --------------------------------------------------------------

def test_streams_and_graphs(ops):
    D, n = 520, 300
    layer, rot = ops.RmsNorm(D), ops.Rotary(40)
    w = 1 + _rand((D,), "f32", 2, 0.1).cuda()
    x, r, dout = (_rand((n, D), "bf16", k).cuda() for k in range(3))
    s = dict(y=torch.empty_like(x), h=torch.empty_like(x), rstd=torch.empty(n, device="cuda"), p=ops.Packed.empty((n, D)),
             a=torch.empty_like(x), pa=ops.Packed.empty((n, D)), da=torch.empty_like(x), dx=torch.empty_like(x),
             dw=torch.empty(D, device="cuda"), q=torch.empty_like(x))

    def go(stream=None):
        layer.forward(x, w, residual=r, summed=s["h"], saved=s["p"], rstd=s["rstd"], out=s["y"], stream=stream)
        rot.forward(s["y"].view(1, n, 13, 40), q_out=s["q"].view(1, n, 13, 40), stream=stream)
        ops.activation(s["q"], kind="silu", out=s["a"], saved=s["pa"], stream=stream)
        ops.activation_backward(dout, s["pa"], kind="silu", dx=s["da"], stream=stream)
        rot.backward(s["da"].view(1, n, 13, 40), q_out=s["da"].view(1, n, 13, 40), stream=stream)
        layer.backward(s["da"], s["p"], s["rstd"], w, residual_grad=dout, out=s["dx"], weight_grad=s["dw"], stream=stream)

    go()
    want = {k: v.clone() for k, v in s.items() if torch.is_tensor(v)}
    clear = lambda: [v.zero_() for v in s.values() if torch.is_tensor(v)]  # noqa: E731
    side = torch.cuda.Stream()
    clear()
    side.wait_stream(torch.cuda.current_stream())
    go(side)  # the stream argument, while another is current
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(s[k], want[k]) for k in want)
    clear()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    other = [v.clone() for v in (x, r, dout)]
    for _ in range(3):
        clear()
        graph.replay()
    assert all(torch.equal(s[k], want[k]) for k in want)
    for v in (x, r, dout):
        v.mul_(0.5)
    graph.replay()
    half = {k: v.clone() for k, v in s.items() if torch.is_tensor(v)}
    go()
    assert all(torch.equal(s[k], half[k]) for k in half) and not torch.equal(half["y"], want["y"])
    for v, o in zip((x, r, dout), other):
        v.copy_(o)
    assert layer.status() == 0


def test_launches_in_a_row_see_each_others_results(ops):
    """Kernels may start before the one before them has ended: a chain without any wait between equals one with them."""
    D, n = 512, 2000
    layer, rot = ops.RmsNorm(D), ops.Rotary(64, interleaved=True)
    w, dw = 1 + _rand((D,), "f32", 2, 0.1).cuda(), torch.zeros(D, device="cuda")
    x0 = _rand((n, D), "bf16", 3).cuda()
    p, pa, rstd, dup = ops.Packed.empty((n, D)), ops.Packed.empty((n, D)), torch.empty(n, device="cuda"), torch.empty_like(x0)

    def go(x, wait):
        w_ = w.clone()
        for _ in range(12):
            for step in (lambda: layer.forward(x, w_, residual=x0, saved=p, rstd=rstd, out=x),
                         lambda: rot.forward(x.view(1, n, 8, 64), q_out=x.view(1, n, 8, 64), first_position=5),
                         lambda: ops.activation(x, x0, kind="gelu", out=x, saved=pa),
                         lambda: ops.unpack8(pa, out=dup),
                         lambda: layer.backward(x, p, rstd, w_, residual_grad=dup, out=x, weight_grad=w_, weight_base=w_),
                         lambda: x.mul_(0.25), lambda: w_.clamp_(0.5, 2.0),
                         lambda: ops.pack8(x, out=pa),
                         lambda: ops.activation_backward(x, pa, kind="silu", dx=x)):
                step()
                if wait:
                    torch.cuda.synchronize()
        return x, w_

    want = go(x0.clone(), True)
    for _ in range(5):
        got = go(x0.clone(), False)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert layer.status() == 0 and bool(want[0].isfinite().all()) and dw.sum() == 0


def test_calls_of_several_host_threads(ops):
    import threading
    D, n = 264, 500
    layer, rot = ops.RmsNorm(D), ops.Rotary(66, rotary_dim=32)
    x = _rand((n, D), "bf16", 3).cuda()
    want = (layer.forward(x), rot.forward(x.view(1, n, 4, 66)), ops.activation(x), ops.unpack8(ops.pack8(x)))
    failed = []

    def work(i):
        try:
            own, stream = ops.RmsNorm(D), torch.cuda.Stream()
            rstd, dw = torch.ones(n, device="cuda"), torch.empty(D, device="cuda")
            stream.wait_stream(torch.cuda.default_stream())
            with torch.cuda.stream(stream):
                for k in range(50):
                    got = (layer.forward(x), rot.forward(x.view(1, n, 4, 66)), ops.activation(x), ops.unpack8(ops.pack8(x)))
                    own.backward(x, x, rstd, weight_grad=dw)
                    bad = ops.Packed.empty((n, D), group=7)
                    try:
                        ops.pack8(x, out=bad)
                        failed.append("no refusal")
                    except ops.LionCubError as e:
                        if "group" not in str(e):
                            failed.append(str(e))
                    stream.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want)):
                        failed.append((i, k))
            assert own.status() == 0
        except Exception as e:  # noqa: BLE001
            failed.append(repr(e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not failed, failed[:3]


def test_waits_that_run_out_and_guards(ops, monkeypatch):
    """The first wait for a row's copies gives up after one test: the call ends, and the status word tells."""
    n, D = 4000, 768
    dout, h, rstd = _rand((n, D), "bf16", 1).cuda(), _rand((n, D), "f32", 2).cuda(), torch.ones(n, device="cuda")
    good = ops.RmsNorm(D)
    dw, want = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    dx = good.backward(dout, h, rstd, weight_grad=want)
    monkeypatch.setenv("LIONCUB_WAIT_POLLS", "1")
    bad = ops.RmsNorm(D)
    monkeypatch.delenv("LIONCUB_WAIT_POLLS")
    bad.backward(dout, h, rstd, weight_grad=dw)
    assert bad.status() == 1  # LIONCUB_STATUS_WAIT_TIMEOUT
    bad.close()
    assert torch.equal(good.backward(dout, h, rstd, weight_grad=dw), dx) and torch.equal(dw, want) and good.status() == 0


def test_offsets_beyond_32_bits(ops):
    """More than 2^32 elements: the first, a middle and the last rows are those of a small call."""
    D, n = 16384, (1 << 18) + 1037
    x = torch.zeros(n, D, dtype=torch.bfloat16, device="cuda")
    few = [0, 1, 131072, 262143, 262144, n - 2, n - 1]
    rows = _rand((len(few), D), "bf16", 4).cuda()
    x[few] = rows
    layer = ops.RmsNorm(D)
    rstd, small = torch.empty(n, device="cuda"), torch.empty(len(few), device="cuda")
    p = ops.pack8(x)
    assert torch.equal(p.codes[few], ops.pack8(rows).codes) and torch.equal(p.scales[few], ops.pack8(rows).scales)
    want = layer.forward(rows, rstd=small)
    dx_want = layer.backward(rows, ops.pack8(rows), small)
    y = layer.forward(x, rstd=rstd)
    assert torch.equal(y[few], want) and torch.equal(rstd[few], small)
    assert torch.equal(layer.backward(x, p, rstd, out=y)[few], dx_want)
    assert torch.equal(ops.activation(x, out=y)[few], ops.activation(rows))
    assert torch.equal(ops.unpack8(p, out=y)[few], ops.unpack8(ops.pack8(rows)))
    rot = ops.Rotary(64)
    at = torch.tensor([few], device="cuda")
    assert torch.equal(rot.forward(x.view(1, n, 256, 64), q_out=y.view(1, n, 256, 64))[0, few],
                       rot.forward(rows.view(1, len(few), 256, 64), positions=at)[0])


def test_failed_allocations_and_launches(ops, monkeypatch):
    E = ops.LionCubError
    monkeypatch.setenv("LIONCUB_FAIL_ALLOC", "1")
    for make in (lambda: ops.RmsNorm(64), lambda: ops.Rotary(64)):
        with pytest.raises(E, match="no device memory"):
            make()
    monkeypatch.delenv("LIONCUB_FAIL_ALLOC")
    x, rstd, dw = _rand((9, 64), "f32", 1).cuda(), torch.ones(9, device="cuda"), torch.zeros(64, device="cuda")
    want = torch.zeros(64, device="cuda")
    ops.RmsNorm(64).backward(x, x.clone(), rstd, weight_grad=want)
    for k in (1, 2):
        monkeypatch.setenv("LIONCUB_FAIL_LAUNCH", str(k))
        layer = ops.RmsNorm(64)
        with pytest.raises(E, match="launch"):
            layer.backward(x, x.clone(), rstd, weight_grad=dw)
        layer.backward(x, x.clone(), rstd, weight_grad=dw)  # the next one is whole
        assert torch.equal(dw, want) and layer.status() == 0
    monkeypatch.setenv("LIONCUB_FAIL_LAUNCH", "1")
    rot = ops.Rotary(64)
    with pytest.raises(E, match="launch"):
        rot.forward(x.view(1, 9, 1, 64))
    rot.forward(x.view(1, 9, 1, 64))


# ---- a run of them together -----------------------------------------------------------------------

@pytest.mark.parametrize("code", [None, "int8", "e4m3"])
def test_block_forward_and_backward(ops, code):
    """Norm, rotary positions on a fused product's heads, attention, residual and norm, a gated activation: gradients
    by hand against autograd in 64 bits; with 8-bit checkpoints against the same graph with the restored values put
    in where the checkpoints are read."""
    torch.manual_seed(5)
    B, S, H, D, F = 2, 24, 4, 128, 192
    n, d = B * S, D // H
    mk = lambda *shape, std=1.0: torch.randn(*shape, dtype=torch.float64, device="cuda") * std  # noqa: E731
    x0, wq, wo = mk(n, D), mk(D, 3 * D, std=D ** -0.5), mk(D, D, std=D ** -0.5)
    w1, w2 = mk(D, 2 * F, std=D ** -0.5), mk(F, D, std=F ** -0.5)
    g1, g2, top = 1 + mk(D, std=0.1), 1 + mk(D, std=0.1), mk(n, D)
    rot, norm1, norm2 = ops.Rotary(d), ops.RmsNorm(D), ops.RmsNorm(D)
    mask = torch.full((S, S), float("-inf"), device="cuda").triu(1)

    def heads(t):
        return t.view(B, S, 3, H, d).unbind(2)

    # by the operators, fp32
    f = lambda t: t.float()  # noqa: E731
    r1, r2 = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    pack = lambda cols: ops.Packed.empty((n, cols), group=32, dtype=CODES[code]) if code else None  # noqa: E731
    p1, p2, pg, pu = pack(D), pack(D), pack(F), pack(F)
    y1 = norm1.forward(f(x0), f(g1), rstd=r1, saved=p1)
    qkv = y1 @ f(wq)
    q, k, v = heads(qkv)
    rot.forward(q, k, q_out=q, k_out=k)
    att = torch.softmax(torch.einsum("bshd,bthd->bhst", q, k) * d ** -0.5 + mask, -1)
    o = torch.einsum("bhst,bthd->bshd", att, v).reshape(n, D)
    h = torch.empty(n, D, device="cuda")
    y2 = norm2.forward(o @ f(wo), f(g2), residual=f(x0), summed=h, rstd=r2, saved=p2)
    both = y2 @ f(w1)
    a = ops.activation(both[:, :F], both[:, F:], kind="silu", saved=pg, saved_up=pu)
    z = h + a @ f(w2)

    dz = f(top)
    again = torch.empty(n, F, device="cuda")
    dboth = torch.empty_like(both)
    ops.activation_backward(dz @ f(w2).t(), pg or both[:, :F], pu or both[:, F:], kind="silu", dx=dboth[:, :F], dup=dboth[:, F:],
                            again=again)
    dw2 = again.t() @ dz
    y2_again, dg2 = torch.empty(n, D, device="cuda"), torch.empty(D, device="cuda")
    dh = norm2.backward(dboth @ f(w1).t(), p2 or h, r2, f(g2), residual_grad=dz, weight_grad=dg2, again=y2_again)
    dw1 = y2_again.t() @ dboth
    dwo = o.t() @ dh
    do = (dh @ f(wo).t()).view(B, S, H, d)
    dqkv = torch.empty(n, 3 * D, device="cuda")
    dq, dk, dv = heads(dqkv)
    dv.copy_(torch.einsum("bhst,bshd->bthd", att, do))
    da = torch.einsum("bshd,bthd->bhst", do, v)
    ds = att * (da - (da * att).sum(-1, keepdim=True)) * d ** -0.5
    dq.copy_(torch.einsum("bhst,bthd->bshd", ds, k))
    dk.copy_(torch.einsum("bhst,bshd->bthd", ds, q))
    rot.backward(dq, dk, q_out=dq, k_out=dk)
    y1_again, dg1 = torch.empty(n, D, device="cuda"), torch.empty(D, device="cuda")
    dx = norm1.backward(dqkv @ f(wq).t(), p1 or f(x0), r1, f(g1), residual_grad=dh, weight_grad=dg1, again=y1_again)
    dwq = y1_again.t() @ dqkv

    # autograd in 64 bits; put(t, packed) has the value of what is saved in the backward pass only
    leaves = [t.clone().requires_grad_() for t in (x0, wq, wo, w1, w2, g1, g2)]
    x_, wq_, wo_, w1_, w2_, g1_, g2_ = leaves
    restored = lambda p: ops.unpack8(p, out_dtype=torch.float32).double()  # noqa: E731

    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, p):
            r = (x.square().mean(1) + 1e-5).rsqrt()
            ctx.save_for_backward(x if p is None else restored(p), r, w)
            return x * r[:, None] * w

        @staticmethod
        def backward(ctx, dout):
            x, r, w = ctx.saved_tensors
            nn, g = x * r[:, None], dout * w
            return r[:, None] * (g - nn * (g * nn).mean(1, keepdim=True)), (dout * nn).sum(0), None

    class Product(torch.autograd.Function):  # its weight's gradient from the input that is computed again
        @staticmethod
        def forward(ctx, x, w, x_again):
            ctx.save_for_backward(x_again, w)
            return x @ w

        @staticmethod
        def backward(ctx, dout):
            x, w = ctx.saved_tensors
            return dout @ w.t(), x.t() @ dout, None

    class Gate(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, u):
            ctx.save_for_backward(*((x, u) if code is None else (restored(pg), restored(pu))))
            return x * torch.sigmoid(x) * u

        @staticmethod
        def backward(ctx, dout):
            x, u = ctx.saved_tensors
            s = torch.sigmoid(x)
            return dout * u * s * (1 + x * (1 - s)), dout * x * s

    def norm_again(x, r, w, p):
        return ((x if p is None else restored(p)) * r[:, None].double() * w).detach()

    def turned(t):
        angle = torch.arange(S, dtype=torch.float64, device="cuda")[:, None] * torch.tensor(rot.frequencies, dtype=torch.float64, device="cuda")
        c, s_ = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
        u, w = t[..., :d // 2], t[..., d // 2:]
        return torch.cat([u * c - w * s_, u * s_ + w * c], -1)

    y_ = Norm.apply(x_, g1_, p1)
    q_, k_, v_ = heads(Product.apply(y_, wq_, norm_again(x_, r1, g1_, p1)))
    q_, k_ = turned(q_), turned(k_)
    att_ = torch.softmax(torch.einsum("bshd,bthd->bhst", q_, k_) * d ** -0.5 + mask.double(), -1)
    o_ = torch.einsum("bhst,bthd->bshd", att_, v_).reshape(n, D)
    h_ = x_ + o_ @ wo_
    y2_ = Norm.apply(h_, g2_, p2)
    both_ = Product.apply(y2_, w1_, norm_again(h_, r2, g2_, p2))
    a_ = Gate.apply(both_[:, :F], both_[:, F:])
    gate_in = (both_[:, :F], both_[:, F:]) if code is None else (restored(pg), restored(pu))
    z_ = h_ + Product.apply(a_, w2_, (gate_in[0] * torch.sigmoid(gate_in[0]) * gate_in[1]).detach())
    z_.backward(top)
    assert (z.double() - z_).abs().max() < 1e-4 * z_.abs().max()
    # fp32 throughout: sums of up to 192 products in 12 steps, each off by some 1e-6 of its size
    for got, leaf in zip((dx, dwq, dwo, dw1, dw2, dg1, dg2), leaves):
        assert (got.double() - leaf.grad).abs().max() < 1e-4 * leaf.grad.abs().max()
    assert norm1.status() == 0 and norm2.status() == 0


def test_bounds_checked_build(ops):
    """The same library with its workspace's indexes checked in the kernels: nothing is recorded."""
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    from communication_compressed_sign_gb300 import build
    lib = build.build(bounds_check=True)
    if os.environ.get("LIONCUB_LIBRARY") == lib:
        return
    r = subprocess.run([sys.executable, "-m", "pytest", "tests/test_gpu_block.py", "-m", "gpu", "-x", "-q", "-p", "no:cacheprovider",
                        "-k", "norm_gradient or streams or block_forward"],
                       cwd=root, env={**os.environ, "LIONCUB_LIBRARY": lib}, capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0 and " passed" in r.stdout, (r.stdout + r.stderr)[-3000:]
