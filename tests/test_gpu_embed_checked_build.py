"""The bounds-checked build of the input-layer operators on batches of every
variant.

In that build the kernels check, before they use them, the rows and columns
that are filled, the places and rows of the walks and of running positions, the
slots of joined sums, the sort's keys, lists and entries, and the lookup's
rows; an index beyond its buffer is skipped and sets the out-of-bounds bit.
The selected tests compare their results and, but for those whose ids are
meant to lie beyond the tables, assert that the status word is 0.
"""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_operators_under_bounds_checks():
    from communication_compressed_sign_gb300 import build
    import __graft_entry__
    __graft_entry__.build()
    lib = build.build(bounds_check=True)
    r = subprocess.run([sys.executable, "-m", "pytest", "tests/test_gpu_embed_batches.py", "tests/test_gpu_embed_order.py",
                        "tests/test_gpu_embed_calls.py", "tests/test_gpu_embed.py", "-m", "gpu", "-x", "-q", "-p",
                        "no:cacheprovider", "-k", "to_the_bit or with_dropout or joined or empty_places or large_repeated or "
                        "running_positions_of or empty_batch or many_sequences"],
                       cwd=ROOT, env={**os.environ, "LIONCUB_LIBRARY": lib}, capture_output=True, text=True, timeout=1200)
    tail = (r.stdout + r.stderr)[-3000:]
    assert r.returncode == 0, tail
    assert " passed" in r.stdout and "failed" not in r.stdout, tail
