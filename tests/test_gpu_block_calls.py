"""Calls of the block operators by tensors of many kinds: views whose rows lie
apart, tensors that carry a tangent, lazily cloned and negated ones, and the
norm's gradient without the weight's."""
import numpy as np
import pytest

from tests import block_reference as ref
from tests.test_gpu_block import CODES, DIMS, EPS, LAYOUTS, T, _check, _np, _packed, _rand, _restored, _strided, _untouched, ops  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def _views():
    a, b = (torch.zeros(s, device="cuda") for s in ((4, 5, 30), (3, 4, 2, 6)))
    for t in (a, b):
        t.copy_(torch.randn(t.shape, generator=torch.Generator().manual_seed(7)))
    return (a[..., :7], a[:, 1:3, :7], a[:, :1, :7], a[:1, :, :7], a[:, ::2, :7], a.transpose(0, 1)[..., :7], a[..., ::2], a[:, :, None, :7],
            a[:1, :1, :7], a[0, :, :9], a[0].t(), a[..., :1], a[:, :, 3:4], a[:, :1].expand(4, 5, 30), b[..., :4], b[:, :, :1, :4],
            b.permute(1, 0, 2, 3)[..., :4], b[:, :, 0], b[:, 1, :, :4], a[0, 0, ::3], a[0, 1:2, :9], a[0, 0, :11], a[:, :, ::30],
            a[2:3, 3:4].expand(1, 1, 30), a[:, :1, :7].expand(4, 1, 7), b[:, ::3, ::1, :5], b[1:2, :, :, :6], b[::2, :1, :1, 1:4])


@pytest.mark.parametrize("number", range(28))
def test_views_as_matrices(ops, number):  # noqa: F811
    """A view is taken for the matrix that torch's own view of it is, or refused where there is none."""
    t = _views()[number]
    cols = t.size(-1)
    n = t.numel() // cols
    try:
        m = t.view(-1, cols)
        want = "columns" if cols > 1 and m.stride(1) != 1 else "stride" if n > 1 and m.stride(0) < cols else None
    except RuntimeError:
        want = "columns|fixed distance"
    if want:
        for call in (lambda: ops.pack8(t), lambda: ops.unpack8(ops.Packed.empty(t.shape), out=t), lambda: ops.activation(t),
                     lambda: ops.RmsNorm(cols).forward(t)):
            with pytest.raises((ValueError, ops.LionCubError), match=want):
                call()
        return
    whole = t.contiguous()
    p, q = ops.pack8(t, group=32), ops.pack8(whole, group=32)
    assert torch.equal(p.codes, q.codes) and torch.equal(p.scales, q.scales)
    assert torch.equal(ops.activation(t, kind="silu"), ops.activation(whole, kind="silu"))
    layer = ops.RmsNorm(cols)
    assert torch.equal(layer.forward(t), layer.forward(whole))
    base = t._base
    elsewhere = base.clone()
    mine = torch.zeros_like(base, dtype=torch.bool)
    inside = mine.as_strided(t.shape, t.stride(), t.storage_offset())
    inside.fill_(True)
    ops.unpack8(q, out=t)  # writes the view, and nothing beside it
    assert torch.equal(t, ops.unpack8(q, out_dtype=torch.float32)) and torch.equal(base[~mine], elsewhere[~mine])


def test_codes_and_scales_in_views(ops):  # noqa: F811
    """Codes and scales of three dimensions out of wider ones."""
    x = _rand((6, 5, 96), "f32", 3).cuda()
    want = ops.pack8(x, group=32)
    codes, scales = torch.full((6, 10, 112), 7, dtype=torch.int8, device="cuda"), torch.full((6, 5, 9), 7.0, device="cuda")
    p = ops.Packed(codes[:, :, :96].unflatten(1, (5, 2))[:, :, 0], scales[..., 2:5], 32)
    ops.pack8(x, out=p)
    assert torch.equal(p.codes, want.codes) and torch.equal(p.scales, want.scales)
    assert torch.equal(ops.unpack8(p), ops.unpack8(want))
    assert (codes[:, 1::2] == 7).all() and (codes[..., 96:] == 7).all() and (scales[..., :2] == 7).all() and (scales[..., 5:] == 7).all()
    for bad in (ops.Packed(codes[:, :5, :96], scales[..., :3], 32), ops.Packed(p.codes, scales[:, :, :6:2], 32),
                ops.Packed(p.codes, scales.transpose(0, 1)[:, :, :3], 32)):
        with pytest.raises(ValueError):
            ops.pack8(x, out=bad)


def _calls(ops):  # noqa: F811
    """(name, call by its tensors, names of its results, other tensors by name): every entry with all of its operands."""
    n, D = 6, 128
    new = lambda *shape: torch.zeros(*(shape or (n, D)), device="cuda")  # noqa: E731
    x, up, dout, w = (_rand((n, D) if k < 3 else (D,), "f32", k).cuda() for k in range(4))
    layer, rot = ops.RmsNorm(D), ops.Rotary(32)
    rstd = (x.double().square().mean(1) + EPS).rsqrt().float()
    kept = ops.pack8(x)
    heads = lambda t: t.view(1, n, 4, 32)  # noqa: E731
    P = lambda c, s: ops.Packed(c, s, 128)  # noqa: E731
    codes = lambda: torch.zeros(n, D, dtype=torch.int8, device="cuda")  # noqa: E731
    return (
        ("norm", lambda x, residual, weight, summed, codes, scales, rstd, out: layer.forward(
            x, weight, residual=residual, summed=summed, saved=P(codes, scales), rstd=rstd, out=out),
         dict(summed=new(), codes=codes(), scales=new(n, 1), rstd=new(n), out=new()), dict(x=x, residual=up, weight=w)),
        ("gradient", lambda dout, saved, rstd, weight, residual_grad, base, out, weight_grad, again: layer.backward(
            dout, saved, rstd, weight, residual_grad=residual_grad, out=out, weight_grad=weight_grad, weight_base=base, again=again),
         dict(out=new(), weight_grad=new(D), again=new()), dict(dout=dout, saved=x, rstd=rstd, weight=w, residual_grad=up, base=w.clone())),
        ("pack8", lambda x, codes, scales: ops.pack8(x, out=P(codes, scales)), dict(codes=codes(), scales=new(n, 1)), dict(x=x)),
        ("unpack8", lambda scales, out: ops.unpack8(P(kept.codes, scales), out=out), dict(out=new()), dict(scales=kept.scales)),
        ("activation", lambda x, up, out, codes, scales: ops.activation(x, up, out=out, saved=P(codes, scales)),
         dict(out=new(), codes=codes(), scales=new(n, 1)), dict(x=x, up=up)),
        ("activation_backward", lambda dout, x, up, dx, dup, again: ops.activation_backward(dout, x, up, dx=dx, dup=dup, again=again),
         dict(dx=new(), dup=new(), again=new()), dict(dout=dout, x=x, up=up)),
        ("rotary", lambda q, k, q_out, k_out: rot.forward(heads(q), heads(k), q_out=heads(q_out), k_out=heads(k_out)),
         dict(q_out=new(), k_out=new()), dict(q=x, k=up)),
    )


@pytest.mark.parametrize("number", range(7))
def test_tensors_with_a_tangent_are_refused(ops, number):  # noqa: F811
    """A forward-mode derivative would be lost, and with it the caller's result."""
    from torch.autograd import forward_ad
    _, call, results, inputs = _calls(ops)[number]
    call(**results, **inputs)
    with forward_ad.dual_level():
        call(**results, **inputs)  # no tensor has one
        for name, t in {**results, **inputs}.items():
            if not t.is_floating_point():
                continue
            dual = {**results, **inputs, name: forward_ad.make_dual(t, torch.ones_like(t))}
            for context in (torch.enable_grad, torch.no_grad):
                with context(), pytest.raises(ValueError, match="tangent"):
                    call(**dual)
            call(**{**dual, name: forward_ad.unpack_dual(dual[name]).primal})
    call(**results, **inputs)


@pytest.mark.parametrize("number", range(7))
def test_lazily_cloned_results(ops, number):  # noqa: F811
    """A result that shares its memory with another tensor until one of them is written: the other keeps its values."""
    _, call, results, inputs = _calls(ops)[number]
    call(**results, **inputs)
    want = {k: t.clone() for k, t in results.items()}
    for name, t in results.items():
        other = torch.full(t.shape, 7.0, device="cuda").to(t.dtype)
        mine = torch._lazy_clone(other)
        call(**{**results, name: mine}, **inputs)
        assert (other == 7).all() and torch.equal(mine, want[name]), name


@pytest.mark.parametrize("number", range(7))
def test_negated_views_are_refused(ops, number):  # noqa: F811
    """Their memory holds other numbers than they do."""
    _, call, results, inputs = _calls(ops)[number]
    for name, t in {**results, **inputs}.items():
        if t.is_floating_point():
            with pytest.raises(ValueError, match="negated"):
                call(**{**results, **inputs, name: torch._neg_view(t)})


@pytest.mark.parametrize("n,D", DIMS + [(700, 771), (1000, 768)])
@pytest.mark.parametrize("dk,hk,gk", [("bf16", "bf16", "bf16"), ("bf16", "int8", "bf16"), ("f32", "f32", "f32"), ("bf16", "f32", None),
                                      ("f32", "e4m3", None)])
def test_norm_gradient_without_the_weights(ops, n, D, dk, hk, gk):  # noqa: F811
    """dx by one launch, against the definition, and to the bit what it is beside a weight's gradient."""
    layer = ops.RmsNorm(D, eps=1e-5)
    for (pad, shift), wk, group in zip(LAYOUTS, ("f32", None, "bf16", "f32", "bf16"), (128, 0, 64, 32, 0)):
        dout, h = _rand((n, D), dk, n * 3 + D), _rand((n, D), "f32" if hk in CODES else hk, D)
        g = None if gk is None else _rand((n, D), gk, D + 2)
        w = None if wk is None else 1 + _rand((D,), "f32", D, 0.3).to(T[wk])
        rstd = (h.double().square().mean(1) + EPS).rsqrt().float()
        if hk in CODES:
            saved, _, _ = _packed(ops, n, D, hk, group, pad, shift)
            ops.pack8(h.cuda(), out=saved)
            exact_h = _restored(saved, hk).astype(np.float64)
        else:
            saved, exact_h = _strided(h, pad, shift)[0], _np(h)
        gv = None if g is None else _strided(g, pad, shift)[0]
        dv, wv = _strided(dout, pad, shift)[0], None if w is None else w.cuda()
        (x0, xm), _, _ = ref.norm_gradient(_np(dout), exact_h, _np(rstd), None if w is None else _np(w), None if g is None else _np(g), None)
        both = []
        for grad in (None, torch.empty(D, device="cuda")):
            dx, whole = _strided(torch.zeros(n, D, dtype=T[gk or "f32"]), pad, shift)
            layer.backward(dv, saved, rstd.cuda(), wv, residual_grad=gv, out=dx, weight_grad=grad)
            _check(dx, x0, xm, 64, dx.dtype)
            _untouched(whole, n, D, pad, shift)
            both.append(dx)
        assert torch.equal(*both)
    assert layer.status() == 0


@pytest.mark.parametrize("D", [1, 64, 771, 2048, 9001, 16384])
def test_one_row_in_the_weights_place(ops, D):  # noqa: F811
    """Results of one row that are the weight (read by then), and the weight's gradient over the weight of any rows."""
    for n in (1, 5):
        x, dout, r, w = (_rand((n, D) if k < 3 else (1, D), "f32", k + D).cuda() for k in range(4))
        layer, rstd = ops.RmsNorm(D), torch.empty(n, device="cuda")
        kept = ops.Packed.empty((n, D))
        y = layer.forward(x, w, residual=r, rstd=rstd, saved=kept)
        saved, dw, again = x + r, torch.empty(D, device="cuda"), torch.empty_like(x)
        dx = layer.backward(dout, saved, rstd, w, residual_grad=r, weight_grad=dw, again=again)
        if n == 1:
            v = w.clone()
            assert torch.equal(layer.forward(x, v, residual=r, out=v), y) and torch.equal(v, y)
            for out, more in ((True, False), (False, True)):
                v, grad, other = w.clone(), torch.empty_like(dw), torch.empty_like(x)
                layer.backward(dout, saved, rstd, v, residual_grad=r, weight_grad=grad, out=v if out else other, again=v if more else other)
                a, b = (v, other) if out else (other, v)
                assert torch.equal(a, dx) and torch.equal(b, again) and torch.equal(grad, dw)
        v = w.clone()
        assert torch.equal(layer.backward(dout, saved, rstd, v, residual_grad=r, weight_grad=v), dx) and torch.equal(v[0], dw)
        v = w.clone()
        layer.backward(dout, saved, rstd, v, weight_grad=v, weight_base=v)
        assert torch.equal(v[0], dw + w[0])
        assert layer.status() == 0
