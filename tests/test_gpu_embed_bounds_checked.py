"""The bounds-checked build of the input-layer operators: every index of the
sort and the row sums is validated in-kernel, and the status word, which each
gradient test reads, must stay 0."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_gradients_under_bounds_checks():
    from communication_compressed_sign_gb300 import build
    import __graft_entry__
    __graft_entry__.build()
    lib = build.build(bounds_check=True)
    r = subprocess.run([sys.executable, "-m", "pytest", "tests/test_gpu_embed.py", "-m", "gpu", "-x", "-q",
                        "-p", "no:cacheprovider", "-k", "repeated or many_sequences or large_vocabulary or empty_batch or beyond_the_tables or packed or flat_vector"],
                       cwd=ROOT, env={**os.environ, "LIONCUB_LIBRARY": lib}, capture_output=True, text=True, timeout=1200)
    tail = (r.stdout + r.stderr)[-3000:]
    assert r.returncode == 0, tail
    assert " passed" in r.stdout and "failed" not in r.stdout, tail
