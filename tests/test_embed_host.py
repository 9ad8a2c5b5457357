"""Host-only checks of the input-layer operators: exported symbols, struct
sizes, argument checks that run before any CUDA call, the header as plain C,
and the reference generator against SplitMix64's published outputs."""
import ctypes
import json
import os
import re
import shutil
import subprocess

import numpy as np
import pytest

from tests import embed_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def em():
    from communication_compressed_sign_gb300 import build
    build.build()
    from communication_compressed_sign_gb300 import embed
    embed.load()
    return embed


def test_symbols_and_struct_sizes(em):
    with open(os.path.join(ROOT, "include", "lioncub_embed.h")) as f:
        declared = sorted(set(re.findall(r"LIONCUB_API[^;(]*?\b(lioncub_\w+)\s*\(", f.read())))
    assert sorted(em.EXPORTED) == declared
    lib = ctypes.CDLL(em.lioncub.LIB_PATH)
    assert all(hasattr(lib, name) for name in declared)
    assert [ctypes.sizeof(t) for t in (em.Rows, em.TokenBatch, em.DropSpec)] == [24, 48, 24]
    assert em._pack_rows(1 << 40, 5, 1, 0) == bytes(em.Rows(1 << 40, 5, 1, 0))
    assert em._pack_batch(1 << 40, 0, 7, 3, 2, 1, 0) == bytes(em.TokenBatch(1 << 40, None, 7, 3, 2, 1, 0))
    assert em._pack_drop(2**64 - 1, 9, 0.25, 0) == bytes(em.DropSpec(2**64 - 1, 9, 0.25, 0))


def test_create_refusals(em):
    L = em.load()
    h = ctypes.c_void_p()
    arg = em.lioncub.ERR_ARG
    assert L.lioncub_embed_create(None, 10, 8, 0, 4, 1.0) == arg
    for vocab, dim, pos, n, scale in ((0, 8, 0, 4, 1.0), (em.MAX_VOCAB + 1, 8, 0, 4, 1.0), (10, 0, 0, 4, 1.0),
                                      (10, em.MAX_DIM + 1, 0, 4, 1.0), (10, 8, -1, 4, 1.0),
                                      (10, 8, em.MAX_VOCAB + 1, 4, 1.0), (10, 8, 0, -1, 1.0),
                                      (10, 8, 0, em.MAX_TOKENS + 1, 1.0), (10, 8, 0, 4, float("nan")),
                                      (10, 8, 0, 4, float("inf"))):
        assert L.lioncub_embed_create(ctypes.byref(h), vocab, dim, pos, n, scale) == arg
        assert h.value is None and L.lioncub_embed_last_error(None)
    assert L.lioncub_embed_forward(None, None, None, None, None, None, None) == arg
    assert L.lioncub_embed_backward(None, None, None, None, None, None, None, None, None) == arg
    assert L.lioncub_embed_status(None, None, None) == arg
    L.lioncub_embed_destroy(None)


def test_dropout_refusals(em):
    """Made-up addresses: every call is refused before anything is launched."""
    L = em.load()
    arg, align = em.lioncub.ERR_ARG, em.lioncub.ERR_ALIGN
    drop = em.DropSpec(1, 2, 0.5, 0)

    def call(rows, cols, x=(4096, None, 1), out=(1 << 20, None, 1), res=None, d=drop):
        r = lambda t: ctypes.byref(em.Rows(t[0], cols if t[1] is None else t[1], t[2], 0))  # noqa: E731
        return L.lioncub_dropout_forward(rows, cols, r(x), r(res) if res else None, r(out), ctypes.byref(d), None)

    assert call(-1, 8) == arg and call(8, -1) == arg and call(1 << 32, 8) == arg and call(1, 1 << 42) == arg
    assert call(8, 8, x=(None, None, 1)) == arg
    assert call(8, 8, x=(4096, 7, 1)) == arg
    assert call(8, 8, x=(4096, None, 2)) == arg
    assert call(8, 8, x=(4098, None, 1)) == align
    assert call(8, 8, out=((1 << 20) + 1, None, 0)) == align
    assert call(8, 8, res=(1 << 21, None, 0)) == arg
    assert b"type" in L.lioncub_embed_last_error(None)
    assert call(8, 8, out=(4096 + 32, None, 1)) == arg and b"overlaps" in L.lioncub_embed_last_error(None)
    # the columns of one buffer side by side do not overlap; one column more does
    assert call(8, 8, x=(4096, 16, 1), out=(4096 + 28, 16, 1)) == arg
    assert call(8, 9, x=(4096, 16, 1), out=(4096 + 32, 16, 1)) == arg
    assert call(8, 9, x=(4096 + 32, 16, 1), out=(4096, 16, 1)) == arg
    assert call(2, 65535 * 256 + 1, x=(4096, 1 << 25, 1), out=(1 << 40, 1 << 25, 1)) == arg
    for p in (-0.5, 1.5, float("nan")):
        assert call(8, 8, d=em.DropSpec(1, 2, p, 0)) == arg
    assert call(0, 8) == 0 and call(8, 0, x=(None, 0, 1), out=(None, 0, 1)) == 0  # nothing to do


def test_reference_generator():
    with open(os.path.join(ROOT, "tests", "golden", "splitmix64_vectors.json")) as f:
        cases = json.load(f)["cases"]
    for c in cases:
        want = c.get("outputs") or [int(v, 16) for v in c["outputs_hex"]]
        assert [int(v) for v in ref.splitmix64(c["seed"], np.arange(len(want)))] == want
    # element e: field e % 4 of output e // 4 of the key (seed 0, stream 0: its first output)
    key = 0xE220A8397B1DCDAF
    z = [int(v) for v in ref.splitmix64(key, np.arange(3))]
    fields = [(z[e // 4] >> (16 * (e % 4))) & 0xFFFF for e in range(10)]
    assert ref.keep_mask(2, 5, (0.5, 0, 0)).reshape(-1).tolist() == [f >= 32768 for f in fields]
    assert ref.keep_mask(4, 5, (1.0, 0, 0)).sum() == 0 and ref.keep_mask(4, 5, None).all()


PROGRAM = r"""
#include "lioncub_embed.h"
#include <stdio.h>

int main(void)
{
    lioncub_embed_t h = 0;
    lioncub_rows m = {0, 8, LIONCUB_ROWS_F32, 0};
    lioncub_drop d = {1, 2, 2.0f, 0};
    int ok = sizeof(lioncub_rows) == 24 && sizeof(lioncub_token_batch) == 48 && sizeof(lioncub_drop) == 24;
    ok = ok && lioncub_embed_create(&h, 0, 8, 0, 4, 1.0f) == LIONCUB_ERR_ARG && h == 0;
    ok = ok && lioncub_dropout_forward(0, 8, &m, 0, &m, &d, 0) == LIONCUB_ERR_ARG;
    ok = ok && lioncub_embed_last_error(0)[0] != 0;
    printf("%s\n", ok ? "OK" : "FAIL");
    return !ok;
}
"""


def test_header_is_c99_and_links(em, tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    (tmp_path / "a.c").write_text(PROGRAM)
    libdir = os.path.dirname(em.lioncub.LIB_PATH)
    r = subprocess.run([cc, "-std=c99", "-pedantic", "-Wall", "-Wextra", "-Werror", f"-I{ROOT}/include",
                        str(tmp_path / "a.c"), f"-L{libdir}", "-llioncub", f"-Wl,-rpath,{libdir}", "-o",
                        str(tmp_path / "a")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(tmp_path / "a")], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "OK"
