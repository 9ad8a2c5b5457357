"""What the input-layer wrappers take and refuse of tensors, on the CPU (whose device number is -1)."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def em():
    from communication_compressed_sign_gb300 import build, embed
    build.build()
    embed._use_torch()
    return embed


def test_tensors_with_a_tangent_are_refused(em):
    """A forward-mode derivative would be lost, and with it the caller's result."""
    from torch.autograd import forward_ad
    t = torch.randn(4, 8)
    want = em._rows(t, "x", 4, 8, -1)
    with forward_ad.dual_level():
        assert em._rows(t, "x", 4, 8, -1) == want
        dual = forward_ad.make_dual(t, torch.ones_like(t))
        for context in (torch.enable_grad, torch.no_grad):
            with context(), pytest.raises(ValueError, match="x has a tangent"):
                em._rows(dual, "x", 4, 8, -1)
        with forward_ad._set_fwd_grad_enabled(False):  # torch itself lets tangents go here
            em._rows(dual, "x", 4, 8, -1)
        assert em._rows(forward_ad.unpack_dual(dual).primal, "x", 4, 8, -1) == want
    assert em._rows(t, "x", 4, 8, -1) == want


def test_negated_views_are_refused(em):
    """Their memory holds other numbers than they do."""
    t = torch.randn(4, 1, dtype=torch.complex64).conj().imag
    assert t.is_neg()
    with pytest.raises(ValueError, match="x is a negated view"):
        em._rows(t, "x", 4, 1, -1)
    assert em._rows(t.resolve_neg(), "x", 4, 1, -1)
