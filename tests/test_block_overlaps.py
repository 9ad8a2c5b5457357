"""Which operands of a block operator may share memory, without a GPU: the C
entries' own code compiled against a stand-in for the CUDA runtime, whose kernels
are counted and not run.  The addresses are made up."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "communication_compressed_sign_gb300", "csrc")

STAND_IN = r"""
#include "block.cu"

static int launches = 0;
static cudaError_t count() { ++launches; return cudaSuccess; }

namespace lc {
cudaError_t launch_guard_check(const GuardList&, int*, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_norm(NormArgs, bool, cudaStream_t) { return count(); }
int norm_grad_blocks(int64_t, int, int) { return 1; }
cudaError_t launch_norm_grad(NormGradArgs, int, bool, cudaStream_t) { return count(); }
cudaError_t launch_weight_grad(const WeightGradArgs&, cudaStream_t) { return count(); }
cudaError_t launch_pack_rows(const TypedRows&, const PackedRows&, int64_t, int, bool, cudaStream_t) { return count(); }
cudaError_t launch_activation(const ActivationArgs&, int, bool, cudaStream_t) { return count(); }
cudaError_t launch_activation_grad(const ActivationArgs&, int, bool, cudaStream_t) { return count(); }
cudaError_t launch_unpack(const PackedRows&, const TypedRows&, int64_t, int64_t, bool, cudaStream_t) { return count(); }
cudaError_t launch_rotary(const RotaryArgs&, int, bool, int, bool, cudaStream_t) { return count(); }
}

extern "C" {
cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) { *v = 4; return cudaSuccess; }
cudaError_t cudaMalloc(void** p, size_t) { *p = (void*)(uintptr_t(1) << 60); return cudaSuccess; }
cudaError_t cudaFree(void*) { return cudaSuccess; }
cudaError_t cudaMemsetAsync(void*, int, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaMemcpyAsync(void*, const void*, size_t, cudaMemcpyKind, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaGetLastError(void) { return cudaSuccess; }
const char* cudaGetErrorName(cudaError_t) { return ""; }
const char* cudaGetErrorString(cudaError_t) { return ""; }
LIONCUB_API int launches_made(void) { return launches; }
}
"""


class Entries:
    """The C functions with what their calls need at hand."""

    def __init__(self, path):
        from communication_compressed_sign_gb300 import block
        self.block, self.lib = block, ctypes.CDLL(path)
        vp, i64 = ctypes.c_void_p, ctypes.c_int64
        L = self.lib
        L.lioncub_rms_norm_create.argtypes = [ctypes.POINTER(vp), i64, ctypes.c_float]
        L.lioncub_rms_norm_forward.argtypes = [vp, i64] + [vp] * 9
        L.lioncub_rms_norm_backward.argtypes = [vp, i64] + [vp] * 11
        L.lioncub_pack8.argtypes = L.lioncub_unpack8.argtypes = [i64, i64, vp, vp, vp]
        L.lioncub_rms_norm_destroy.argtypes = [vp]
        L.lioncub_rms_norm_destroy.restype = None
        L.lioncub_block_last_error.restype = ctypes.c_char_p

    def rows(self, at, cols, kind=1, stride=None):
        return None if at is None else ctypes.byref(self.block.embed.Rows(at, cols if stride is None else stride, kind, 0))

    def packed(self, codes, scales, cols, group=128):
        return ctypes.byref(self.block.PackedRows(codes, scales, cols, -(-cols // group) if group else 1, group, 0))

    def went(self, rc, launches):
        """Whether a call went through (True) or was refused for an overlap (False), and launched as it should."""
        assert rc in (0, self.block.embed.lioncub.ERR_ARG), rc
        if rc:
            assert b"overlaps" in self.lib.lioncub_block_last_error()
        assert self.lib.launches_made() - self.before == (0 if rc else launches)
        return rc == 0

    def forward(self, n, dim, x, out, residual=None, weight=None, summed=None, saved=None, rstd=None, packed_out=None):
        h, L = ctypes.c_void_p(), self.lib
        assert L.lioncub_rms_norm_create(ctypes.byref(h), dim, 1e-5) == 0
        self.before = L.launches_made()
        r = lambda at: self.rows(at, dim)  # noqa: E731
        rc = L.lioncub_rms_norm_forward(h, n, r(x), r(residual), r(weight), r(summed), saved, rstd, r(out), packed_out, None)
        L.lioncub_rms_norm_destroy(h)
        return self.went(rc, 1)

    def backward(self, n, dim, dout, saved, rstd, dx, weight=None, residual_grad=None, base=None, grad=None, again=None):
        h, L = ctypes.c_void_p(), self.lib
        assert L.lioncub_rms_norm_create(ctypes.byref(h), dim, 1e-5) == 0
        self.before = L.launches_made()
        r = lambda at: self.rows(at, dim)  # noqa: E731
        rc = L.lioncub_rms_norm_backward(h, n, r(dout), r(saved), None, rstd, r(weight), r(residual_grad), r(dx), r(base), r(grad),
                                         r(again), None)
        L.lioncub_rms_norm_destroy(h)
        return self.went(rc, 2 if grad else 1)

    def pack(self, rows, cols, x, p):
        self.before = self.lib.launches_made()
        return self.went(self.lib.lioncub_pack8(rows, cols, self.rows(x, cols), p, None), 1)


@pytest.fixture(scope="module")
def entries(tmp_path_factory):
    from communication_compressed_sign_gb300 import build
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    build.build()
    folder = tmp_path_factory.mktemp("entries")
    (folder / "entries.cpp").write_text(STAND_IN)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    r = subprocess.run([cxx, "-std=c++17", "-O1", "-fPIC", "-shared", "-fvisibility=hidden", f"-I{CSRC}", f"-I{build.INCLUDE}", f"-I{cuda}",
                        str(folder / "entries.cpp"), "-o", str(folder / "entries.so"), "-ldl"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return Entries(str(folder / "entries.so"))


# Places of up to 1 MB, which do not overlap.
A, B, C, D, E, F, G = ((k + 1) << 20 for k in range(7))


@pytest.mark.parametrize("n", [1, 5])
def test_a_gradient_may_take_its_inputs_places(entries, n):
    """dx and again over inputs that are read row by row, the weight's gradient over its base: as documented."""
    back = entries.backward
    for dx, again in ((A, None), (A, B), (B, A), (D, A), (D, B), (G, D)):
        assert back(n, 64, A, B, C, dx, residual_grad=D, base=E, grad=E, again=again)
    assert back(n, 64, A, B, C, D, weight=F, base=E, grad=F)  # the weight has been read by then
    assert not back(n, 64, A, B, C, D, again=D)


@pytest.mark.parametrize("n", [1, 5])
def test_what_is_added_to_the_weights_gradient_is_no_result_of_the_rows(entries, n):
    """It is read by the second launch, after the first has written dx and again."""
    back = entries.backward
    assert not back(n, 64, A, B, C, D, base=D, grad=E)
    assert not back(n, 64, A, B, C, D, base=G, grad=E, again=G)
    assert not back(n, 64, A, B, C, D, weight=E, base=E, grad=F, again=E)
    assert not back(n, 1, A, B, C, D, base=D, grad=E)
    assert back(n, 64, A, B, C, D, weight=E, base=E, grad=F)  # two inputs


@pytest.mark.parametrize("n", [1, 5])
def test_the_norms_weight_is_no_sum(entries, n):
    """The weight of one row's norm is read after the sum is written, but before the result is."""
    go = entries.forward
    assert not go(n, 64, A, B, weight=C, summed=C)
    assert not go(n, 64, A, B, residual=D, weight=C, summed=C)
    assert go(1, 64, A, C, weight=C) and not go(5, 64, A, C, weight=C)
    for x, out, residual, summed in ((A, A, None, None), (A, A, B, B), (A, B, B, A), (A, C, B, B), (A, C, B, A), (A, B, None, A)):
        assert go(n, 64, x, out, residual=residual, summed=summed, weight=F)
    assert not go(n, 64, A, B, summed=B)


@pytest.mark.parametrize("n", [1, 5, 64])
def test_a_vector_is_no_matrix(entries, n):
    """rstd has a number for each row, a weight one for each column: with as many of both they are still not one matrix."""
    for dim in (n, n + 1):
        assert not entries.forward(n, dim, A, B, weight=C, rstd=C)
        assert not entries.backward(n, dim, A, B, C, D, grad=C)
    assert not entries.forward(1, 1, A, B, rstd=A)
    assert not entries.backward(1, 1, A, B, C, C)
    assert entries.forward(n, n, A, B, weight=C, rstd=D)


def test_scales_and_codes_are_no_matrix(entries):
    """Scales may lie like a column of fp32, and codes like bytes, but neither is the matrix that is packed."""
    for rows in (1, 7):
        assert not entries.pack(rows, 1, A, entries.packed(B, A, 1))
        assert not entries.pack(rows, 1, A, entries.packed(B, A, 1, group=0))
        assert not entries.pack(rows, 1, A, entries.packed(A, B, 1))
        assert entries.pack(rows, 1, A, entries.packed(B, C, 1))
        assert not entries.forward(rows, 1, A, B, weight=C, saved=entries.packed(D, A, 1))
        assert not entries.forward(rows, 1, A, B, residual=E, saved=entries.packed(D, E, 1))
    assert not entries.forward(1, 1, A, B, weight=C, saved=entries.packed(D, C, 1))
    assert not entries.forward(1, 1, A, None, weight=C, packed_out=entries.packed(D, C, 1))
