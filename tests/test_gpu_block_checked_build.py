"""The block operators in the bounds-checked build, whose kernels compare the row,
columns, group and alignment of every access with the operands' sizes, and those
of the gradient's ring with its slots, and leave out what lies outside."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    from communication_compressed_sign_gb300 import build
    import __graft_entry__
    __graft_entry__.build()
    return build.build(bounds_check=True)


def _run(lib, *args, **env):
    r = subprocess.run([sys.executable, *args], cwd=ROOT, env={**os.environ, "LIONCUB_LIBRARY": lib, **env}, capture_output=True,
                       text=True, timeout=1200)
    assert r.returncode == 0, (r.stdout + r.stderr)[-3000:]
    return r.stdout


def test_every_form_stays_inside(lib):
    """The operators' tests; the one of the ordinary build's own rerun is left out."""
    out = _run(lib, "-m", "pytest", "tests/test_gpu_block.py", "tests/test_gpu_block_calls.py", "-m", "gpu", "-x", "-q", "-p",
               "no:cacheprovider", "-p", "tests.block_checked", "--deselect", "tests/test_gpu_block.py::test_bounds_checked_build")
    assert " passed" in out and "failed" not in out, out[-3000:]


# Matrices of which the kernels are told fewer rows than there are: the rest is recorded, and not written.
FEWER = r"""
import torch
import communication_compressed_sign_gb300 as ops
from tests.block_checked import recorded

n, few, OUT_OF_BOUNDS = 9, 3, 2
for D, dtype, pad in ((64, torch.bfloat16, 64), (64, torch.float32, 64), (77, torch.bfloat16, 3), (77, torch.float32, 3), (2304, torch.float32, 8)):
    new = lambda d=D, t=dtype: torch.full((n, d + pad), 7.0, device="cuda").to(t)[:, :d]
    x, up, dout = (new().normal_() for _ in range(3))
    w, rstd = torch.ones(D, device="cuda"), torch.ones(n, device="cuda")
    def packed(group=32):
        groups = -(-D // group) if group else 1
        return ops.Packed(new(D, torch.int8), new(groups, torch.float32), group)
    ready, ready_up, whole_row = packed(), packed(), packed(0)
    ready.codes.fill_(1), ready_up.codes.fill_(1)
    layer = ops.RmsNorm(D)

    def check(name, call, *results):
        before = [t.clone() for t in results]
        call()
        assert recorded() == OUT_OF_BOUNDS, (name, D, dtype)
        assert recorded() == 0
        for t, b in zip(results, before):
            assert torch.equal(t[few:], b[few:]) and not torch.equal(t[:few], b[:few]), (name, D, dtype)

    a, b, c, p, q = new(), new(), new(), packed(), packed()
    check("norm", lambda: layer.forward(x, w, residual=up, summed=a, saved=p, out=b), a, b, p.codes, p.scales)
    check("norm, codes", lambda: layer.forward(x, out=whole_row), whole_row.codes, whole_row.scales)
    a, b, c, p, q, r = new(), new(), new(), packed(), packed(), packed(0)
    check("pack8", lambda: ops.pack8(x, out=p), p.codes, p.scales)
    check("pack8, rows", lambda: ops.pack8(x, out=r), r.codes, r.scales)
    a.fill_(5.0)  # the codes stand for 1 * 7, which is what new matrices hold
    check("unpack8", lambda: ops.unpack8(ready, out=a), a)
    a, p = new(), packed()
    check("activation", lambda: ops.activation(x, up, out=a, saved=p, saved_up=q), a, p.codes, p.scales, q.codes, q.scales)
    a = new()
    check("gradient", lambda: ops.activation_backward(dout, x, up, dx=a, dup=b, again=c), a, b, c)
    a, b, c = new(), new(), new()
    check("gradient, codes", lambda: ops.activation_backward(dout, ready, ready_up, dx=a, dup=b, again=c), a, b, c)
    for saved in (x, ready):
        a, b = new().fill_(5.0), new().fill_(5.0)
        check("norm's gradient", lambda: layer.backward(dout, saved, rstd, w, residual_grad=up, out=a, again=b, weight_grad=torch.empty_like(w)), a, b)
for dim, part, inter, dtype in ((64, 64, False, torch.bfloat16), (80, 40, True, torch.float32), (66, 22, False, torch.bfloat16), (96, 20, True, torch.float32)):
    rot = ops.Rotary(dim, rotary_dim=part, interleaved=inter)
    q, out = torch.ones(1, n, 4, dim, device="cuda", dtype=dtype), torch.full((1, n, 4, dim), 7.0, device="cuda", dtype=dtype)
    rot.forward(q[:, :, :2], q[:, :, 2:], q_out=out[:, :, :2], k_out=out[:, :, 2:], first_position=3)
    assert recorded() == OUT_OF_BOUNDS and (out[:, few:] == 7).all() and (out[:, :few] != 7).all()
print("found all")
"""


def test_what_lies_outside_is_found(lib):
    assert "found all" in _run(lib, "-c", FEWER, LIONCUB_CHECKED_ROWS="3")


def test_the_ordinary_build_has_no_checks(lib):
    """... and touches all rows whatever the checks' variable says."""
    from communication_compressed_sign_gb300 import build
    out = _run(build.LIB, "-c", "import torch, communication_compressed_sign_gb300 as ops\n"
               "from communication_compressed_sign_gb300 import block\n"
               "x = torch.ones(9, 64, device='cuda')\nassert (ops.unpack8(ops.pack8(x), out_dtype=x.dtype) == 1).all()\n"
               "print(hasattr(block.load(), 'lioncub_block_checked_word'))", LIONCUB_CHECKED_ROWS="3")
    assert out.strip() == "False"
