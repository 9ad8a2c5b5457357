"""Batches of the sizes that training runs: lookups whose warps take several
places and several rounds of them, and running positions whose places are
shared by several warps, with and without dropout.

Lookups are compared bit for bit with the same fp32 operations of torch, each
of which rounds once.  Gradients add small integers and p == 1/2 rescales by
exactly 2, so every fp32 sum is exact in any order.
"""
import itertools

import numpy as np
import pytest

from tests import embed_reference as ref
from tests.test_gpu_embed import T, _rand, ops  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

FIRST = 5

# kind, places of a sequence, places, columns.  A warp takes 4 running places (of
# as many sequences), 2 given ones or 4 without positions once a batch has more
# than 1216 (place, slab of 256 or 224 columns) pairs, and up to 8 rounds of them
# in larger ones; the last sequence is cut short in most.
BATCHES = [
    ("running", 64, 7 * 64 + 37, 520),        # 1 round, 8 sequences
    ("running", 1, 3000, 24),
    ("running", 5000, 3000, 24),              # one sequence, longer than the batch
    ("running", 300, 23 * 300 - 41, 771),     # 2 rounds
    ("running", 1024, 37 * 1024 - 100, 264),  # 4 rounds
    ("running", 1000, 101 * 1000 - 41, 24),   # 8 rounds, 101 sequences for 32 a warp
    ("running", 4000, 25 * 4000 - 10, 13),    # 8 rounds, fewer sequences than a warp could take
    ("given", 50, 3001, 264), ("given", 50, 1300, 771),
    ("given", 50, 13001, 24),                 # 2 rounds
    ("given", 50, 50001, 13),                 # 8 rounds
    ("none", 50, 3001, 264), ("none", 50, 1300, 771),
    ("none", 50, 30001, 24),                  # 2 rounds
    ("none", 50, 90001, 13),                  # 8 rounds
]


def _places(kind, S, n, V, P, index, seed):
    g = np.random.default_rng(seed)
    tok = g.integers(0, V, n)
    tok[g.random(n) < 0.2] = V // 3
    tok[g.random(n) < 0.1] = -1
    tok[n // 2:n // 2 + 9] = -1
    pos = np.arange(n) % S + FIRST if kind == "running" else g.integers(0, P, n)
    return tuple(torch.from_numpy(v).to(index).cuda() for v in (tok, pos))


@pytest.mark.parametrize("kind,S,n,D", BATCHES)
@pytest.mark.parametrize("p", [0.0, 0.1])
def test_lookups_to_the_bit(ops, kind, S, n, D, p):
    V, P = 700, min(S, n) + FIRST + 2
    drop = ops.Drop(p, 11, n) if p else None
    keep = torch.from_numpy(ref.keep_mask(n, D, drop)).cuda()
    r = float(np.float32(ref.rescale(drop)))
    for (tk, ok), index in zip(itertools.product(T, T), itertools.cycle([torch.int64, torch.int32])):
        scale = 1.7 if tk == ok else 1.0
        tok, pos = _places(kind, S, n, V, P, index, n + D)
        table, wpe = _rand((V, D), tk, 1).cuda(), _rand((P, D), tk, 2).cuda()
        layer = ops.TokenEmbedding(V, D, n, positions=P, scale=scale)
        whole = torch.full((n, D + 8), 777.0, dtype=T[ok], device="cuda")
        out = whole[:, :D]
        layer.forward(tok, table, None if kind == "none" else wpe, positions=pos if kind == "given" else None, seq_len=S,
                      first_position=FIRST if kind == "running" else 0, drop=drop, out=out)
        y = table.float()[tok.long().clamp(min=0)] * float(np.float32(scale))
        if kind != "none":
            y = y + wpe.float()[pos.long()]
        want = torch.where(keep & (tok >= 0)[:, None], y * r, torch.zeros_like(y)).to(T[ok])
        assert torch.equal(out, want), (tk, ok)
        assert (whole[:, D:] == 777.0).all(), "wrote outside its matrix"
        assert layer.status() == 0
        layer.close()


@pytest.mark.parametrize("Q,S", [(33, 5), (64, 17), (65, 7), (129, 16), (257, 3), (1000, 9), (1025, 2), (40, 3000)])
@pytest.mark.parametrize("D,dtype", [(264, torch.bfloat16), (771, torch.bfloat16), (24, torch.float32), (77, torch.float32)])
def test_running_positions_with_dropout(ops, Q, S, D, dtype):
    """More than 32 sequences share their positions' sums among warps (up to 1024; above, positions are sorted)."""
    n, V, P = Q * S - S // 2, 13, S + FIRST + 2
    tok, pos = _places("running", S, n, V, P, torch.int64, n)
    g = np.random.default_rng(D)
    dout = g.integers(-2, 3, (n, D)).astype(np.float64)
    drop = ops.Drop(0.5, 21, n)
    keep = ref.keep_mask(n, D, drop)
    layer = ops.TokenEmbedding(V, D, n, positions=P)
    grad, pos_grad = (torch.full((rows, D), float("nan"), device="cuda") for rows in (V, P))
    layer.backward(tok, torch.from_numpy(dout).to(dtype).cuda(), grad, pos_grad=pos_grad, seq_len=S, first_position=FIRST,
                   drop=drop)
    there = tok.cpu().numpy() >= 0
    kept = 2.0 * np.where(keep, dout, 0.0)[there]
    for got, keys, rows in ((grad, tok, V), (pos_grad, pos, P)):
        want = np.zeros((rows, D))
        np.add.at(want, keys.cpu().numpy()[there], kept)
        assert np.array_equal(got.cpu().numpy(), want)
    assert layer.status() == 0
    layer.close()
