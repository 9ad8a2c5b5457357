"""The input-layer operators on the GPU against their definitions in 64 bits.

Bounds are derived, not fitted: a lookup rounds at most 4 times (product, sum,
rescaling, and the rescaling factor itself), a gradient of n places at most
n + 3 times in whatever order they are added (n - 1 additions, two factors
and their product, the base), each rounding at most 2^-24 of the sum of
magnitudes; a bf16 result must lie between the limits of that range rounded to
bf16.  The mask must be equal bit for bit, and zeros must be zeros.
"""
import itertools

import numpy as np
import pytest

from tests import embed_reference as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

T = {"f32": torch.float32, "bf16": torch.bfloat16}


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


def _strided(x, pad, shift=0):
    """The same matrix on the GPU in rows `pad` elements apart, `shift` elements
    into their buffer, the rest poisoned; returns (view, whole buffer)."""
    rows, cols = x.shape
    whole = torch.full((rows * (cols + pad) + shift + 16,), 777.0, dtype=x.dtype, device="cuda")
    view = whole[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    view.copy_(x)
    return view, whole


def _np(x):
    return x.detach().double().cpu().numpy()


def _check(got, exact, magnitude, terms, dtype):
    got = _np(got).reshape(exact.shape)
    low, high = (_np(torch.from_numpy(v).to(T[dtype])) for v in ref.limits(exact, magnitude, terms))
    bad = ~((low <= got) & (got <= high))
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside their limits, first at {np.argwhere(bad)[:4].tolist()}"


# ---- dropout ------------------------------------------------------------------

SHAPES = [(1, 1), (1, 7), (3, 8), (5, 77), (788, 192), (64, 768), (33, 771), (1, 100003), (257, 2049)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("p", [0.1, 0.5])
def test_mask_is_the_generators(ops, rows, cols, p):
    drop = ops.Drop(p, 2**63 + 12345, 2**40 + 3)
    want = ref.keep_mask(rows, cols, drop)
    for kind in T:
        for pad, shift in ((0, 0), (8, 0), (5, 0), (0, 3), (0, 8)):
            x, _ = _strided(torch.ones(rows, cols, dtype=T[kind]), pad, shift)
            assert np.array_equal(_np(ops.dropout(x, drop)) != 0, want), (kind, pad, shift)
            assert np.array_equal(_np(ops.dropout_backward(x, drop)) != 0, want), (kind, pad, shift)
    if rows * cols > 10000:  # five standard deviations of a binomial share
        n = rows * cols
        share = ref.threshold(p) / 65536
        assert abs((~want).mean() - share) < 5 * np.sqrt(share * (1 - share) / n)


@pytest.mark.parametrize("xk,ok", list(itertools.product(T, T)))
@pytest.mark.parametrize("pads", [(0, 0, 0, 0), (8, 16, 0, 0), (5, 0, 3, 0), (0, 0, 0, 1), (3, 3, 3, 2)])
@pytest.mark.parametrize("residual", [False, True])
def test_dropout_values(ops, xk, ok, pads, residual):
    drop = ops.Drop(0.3, 5, 11)
    for rows, cols in ((1, 1), (7, 24), (31, 77), (65, 768)):
        x = _rand((rows, cols), xk, rows)
        r = _rand((rows, cols), ok, rows + 1)
        xv, _ = _strided(x, pads[0], pads[3])
        rv, _ = _strided(r, pads[2], pads[3])
        out, whole = _strided(torch.zeros(rows, cols, dtype=T[ok]), pads[1], pads[3])
        y = ops.dropout(xv, drop, residual=rv if residual else None, out=out)
        keep = ref.keep_mask(rows, cols, drop)
        exact = np.where(keep, _np(x) * ref.rescale(drop), 0.0)
        mag = np.abs(exact)
        if residual:
            exact, mag = exact + _np(r), mag + np.abs(_np(r))
        _check(y, exact, mag, 3, ok)
        if not residual:
            assert (_np(y)[~keep] == 0).all()
        poison = whole.clone()
        poison[pads[3]:pads[3] + rows * (cols + pads[1])].view(rows, -1)[:, :cols] = 777.0
        assert (poison == 777.0).all(), "wrote outside its matrix"


def test_dropout_edges(ops):
    x = torch.tensor([[float("nan"), float("inf"), -float("inf"), 1e38] * 64], device="cuda")
    drop = ops.Drop(0.5, 1, 2)
    keep = torch.from_numpy(ref.keep_mask(1, 256, drop)).cuda()
    y = ops.dropout(x, drop)
    assert (y[~keep] == 0).all()
    want = x * 2
    assert torch.equal(torch.nan_to_num(y[keep]), torch.nan_to_num(want[keep])) and torch.equal(y[keep].isnan(), want[keep].isnan())
    assert (ops.dropout(x, ops.Drop(1.0, 1, 2)) == 0).all()
    r = _rand((1, 256), "f32", 3).cuda()
    assert torch.equal(ops.dropout(x, ops.Drop(1.0, 1, 2), residual=r), r)
    z = _rand((3, 77), "bf16", 4).cuda()
    for none in (None, ops.Drop(0.0, 1, 2), ops.Drop(2.0**-18, 1, 2)):
        assert torch.equal(ops.dropout(z, none), z)
    assert ops.dropout(torch.empty(0, 77, device="cuda"), drop).shape == (0, 77)
    assert ops.dropout(torch.empty(5, 0, device="cuda"), drop).shape == (5, 0)
    # in place on x, on the residual, and between two halves of the same rows
    want = ops.dropout(z, drop)
    c = z.clone()
    assert torch.equal(ops.dropout(c, drop, out=c), want) and torch.equal(c, want)
    c = r.clone()
    assert torch.equal(ops.dropout(r, drop, residual=c, out=c), ops.dropout(r, drop, residual=r))
    both = torch.zeros(3, 154, dtype=torch.bfloat16, device="cuda")
    both[:, :77] = z
    ops.dropout(both[:, :77], drop, out=both[:, 77:])
    assert torch.equal(both[:, 77:], want) and torch.equal(both[:, :77], z)
    # another stream or seed is another mask, the same is the same
    assert torch.equal(ops.dropout(z, drop), want)
    big = torch.ones(64, 768, device="cuda")
    masks = [ops.dropout(big, ops.Drop(0.5, s, t)) != 0 for s, t in ((1, 2), (2, 1), (1, 3), (3, 2))]
    for a, b in itertools.combinations(masks, 2):
        assert 0.45 < (a == b).float().mean().item() < 0.55


def test_dropout_of_a_dimension_beyond_32_bits_of_bytes(ops):
    """Element numbers past 2^32: 65537 x 65544 bf16 elements (8.6 GB), the last rows checked."""
    rows, cols = 65537, 65544
    x = torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda")
    drop = ops.Drop(0.25, 9, 1)
    ops.dropout(x, drop, out=x)
    n = rows * cols
    first = (n - 4096) // 4 * 4
    key = int(ref.splitmix64(9, np.array([1], dtype=np.uint64))[0])
    z = ref.splitmix64(key, np.arange(first // 4, (n + 3) // 4, dtype=np.uint64))
    fields = ((z[:, None] >> np.array([0, 16, 32, 48], dtype=np.uint64)) & np.uint64(0xFFFF)).reshape(-1)[:n - first]
    assert np.array_equal(_np(x.view(-1)[first:]) != 0, fields >= np.uint64(16384))


# ---- lookup -----------------------------------------------------------------------

def _batch(B, S, V, seed, ragged, index, npos, kind):
    rng = np.random.default_rng(seed)
    tok = rng.integers(0, V, (B, S))
    if V > 4:
        tok[rng.random((B, S)) < 0.3] = V // 3  # one frequent token
    if ragged:
        for b in range(B):
            tok[b, rng.integers(0, S + 1):] = -1
    pos = None
    if kind == "packed":
        pos = np.arange(S)[None, :].repeat(B, 0) % rng.integers(1, npos + 1, (B, 1)) % npos
    to = torch.int64 if index == "i64" else torch.int32
    return (torch.from_numpy(tok).to(to).cuda(), None if pos is None else torch.from_numpy(pos).to(to).cuda())


CASES = [
    # B, S, V, D, P, positions
    (1, 1, 1, 1, 1, "run"), (1, 1, 50257, 768, 1024, "run"), (8, 1, 1000, 768, 64, "run"), (3, 17, 65, 8, 32, "packed"),
    (2, 33, 1003, 771, 40, "packed"), (4, 100, 300, 192, 197, "run"), (1, 257, 7, 2048, 300, "none"),
    (5, 64, 513, 77, 64, "run"), (2, 50, 1000, 2056, 50, "packed"), (1, 40, 131075, 16, 0, "none"),
]


@pytest.mark.parametrize("B,S,V,D,P,kind", CASES)
@pytest.mark.parametrize("tk,ok", list(itertools.product(T, T)))
@pytest.mark.parametrize("p", [0.0, 0.1])
def test_lookup(ops, B, S, V, D, P, kind, tk, ok, p):
    seed = B * 1000 + S
    drop = ops.Drop(p, 77, seed) if p else None
    for index, ragged, pad, shift in (("i64", False, 0, 0), ("i32", True, 8, 0), ("i64", True, 5, 3)):
        tok, pos = _batch(B, S, V, seed, ragged, index, P, kind)
        table, wpe = _rand((V, D), tk, seed), _rand((P, D), tk, seed + 1) if kind != "none" else None
        layer = ops.TokenEmbedding(V, D, B * S, positions=P, scale=3.7)
        tv, _ = _strided(table, pad, shift)
        pv = _strided(wpe, pad, shift)[0] if wpe is not None else None
        out, whole = _strided(torch.zeros(B * S, D, dtype=T[ok]), pad, shift)
        first = 0 if kind != "run" else P - S
        if kind == "run" and S > P:
            pytest.skip("longer than the table")
        layer.forward(tok, tv, pv, positions=pos, first_position=first, drop=drop, out=out)
        exact, mag = ref.lookup(tok.cpu().numpy(), _np(table), None if wpe is None else _np(wpe),
                                float(np.float32(3.7)), drop, None if pos is None else pos.cpu().numpy(), S, first)
        _check(out, exact, mag, 4, ok)
        assert (_np(out)[exact == 0] == 0).all() or (mag[exact == 0] > 0).any()
        poison = whole.clone()
        poison[shift:shift + B * S * (D + pad)].view(B * S, -1)[:, :D] = 777.0
        assert (poison == 777.0).all(), "wrote outside its matrix"
        assert layer.status() == 0
        if p and kind == "run" and not ragged:  # a lookup with dropout is a lookup followed by dropout
            plain = layer.forward(tok, tv, pv, first_position=first, out_dtype=torch.float32)
            fused = layer.forward(tok, tv, pv, first_position=first, drop=drop, out_dtype=torch.float32)
            assert torch.equal(fused, ops.dropout(plain.view(B * S, D), drop).view_as(fused))
        layer.close()


def test_lookup_is_fp32_to_the_bit(ops):
    """Each operation rounds once in fp32 and the result once to bf16."""
    tok = torch.arange(100, device="cuda").view(4, 25)
    table, wpe = _rand((100, 768), "f32", 1).cuda(), _rand((25, 768), "f32", 2).cuda()
    layer = ops.TokenEmbedding(100, 768, 100, positions=25, scale=1.7)
    drop = ops.Drop(0.1, 3, 4)
    keep = torch.from_numpy(ref.keep_mask(100, 768, drop)).cuda().view(4, 25, 768)
    r = float(np.float32(65536.0 / (65536.0 - ref.threshold(0.1))))
    y = table[tok] * float(np.float32(1.7)) + wpe[None]
    want = torch.where(keep, y * r, torch.zeros_like(y))
    assert torch.equal(layer.forward(tok, table, wpe, drop=drop, out_dtype=torch.float32), want)
    assert torch.equal(layer.forward(tok, table, wpe, drop=drop), want.to(torch.bfloat16))


@pytest.mark.parametrize("index", [torch.int64, torch.int32])
def test_ids_beyond_the_tables(ops, index):
    V, P, D = 50, 10, 24
    tok = torch.tensor([0, 49, 50, -1, 7, 2**31 - 1, 7], dtype=index, device="cuda")
    pos = torch.tensor([0, 10, 1, 2, -1, 3, 9], dtype=index, device="cuda")
    if index == torch.int64:
        tok[5] = 2**40 + 3
    table, wpe = _rand((V, D), "f32", 1), _rand((P, D), "f32", 2)
    dout = _rand((7, D), "f32", 3)
    layer = ops.TokenEmbedding(V, D, 7, positions=P)
    out = layer.forward(tok, table.cuda(), wpe.cuda(), positions=pos, out_dtype=torch.float32)
    exact, mag = ref.lookup(tok.cpu().numpy(), _np(table), _np(wpe), 1.0, None, pos.cpu().numpy())
    _check(out, exact, mag, 4, "f32")
    assert layer.status() == 8
    layer = ops.TokenEmbedding(V, D, 7, positions=P)
    g, pg = torch.full((V, D), 5.0, device="cuda"), torch.full((P, D), 5.0, device="cuda")
    layer.backward(tok, dout.cuda(), g, pos_grad=pg, positions=pos)
    (e, m, c), (pe, pm, pc) = ref.gradients(tok.cpu().numpy(), V, P, _np(dout), 1.0, None, positions=pos.cpu().numpy())
    _check(g, e, m, c + 3, "f32")
    _check(pg, pe, pm, pc + 3, "f32")
    assert layer.status() == 8


# ---- gradient ----------------------------------------------------------------------

def _gradient(ops, tok, pos, V, D, P, dk, gk, *, first=0, drop=None, base=None, pad=0, shift=0, scale=1.3, want_pos=True,
              nan_empty=False, layer=None):
    B, S = tok.shape
    n = B * S
    dout = _rand((n, D), dk, n + D)
    exact_dout = _np(dout)
    if nan_empty:
        dout[(tok.reshape(-1) < 0).cpu()] = float("nan")
        exact_dout = np.where((tok.reshape(-1) < 0).cpu().numpy()[:, None], 0.0, exact_dout)
    own = layer is None
    layer = layer or ops.TokenEmbedding(V, D, n, positions=P, scale=scale)
    start = _rand((V, D), gk, 5)
    pstart = _rand((max(P, 1), D), gk, 6)
    dv, _ = _strided(dout, pad, shift)
    gv, whole = _strided(start, pad, shift)
    pgv, pwhole = _strided(pstart, pad, shift)
    want_pos = want_pos and P > 0
    more = {}
    if base == "in place":
        more = dict(base=gv, pos_base=pgv if want_pos else None)
    elif base == "other":
        more = dict(base=_strided(start, pad, shift)[0], pos_base=_strided(pstart, pad, shift)[0] if want_pos else None)
        gv.fill_(float("nan"))
        pgv.fill_(float("nan"))
    layer.backward(tok, dv if pad or shift else dv.view(B, S, D), gv, pos_grad=pgv if want_pos else None, positions=pos,
                   first_position=first, drop=drop, **more)
    t, q = ref.gradients(tok.cpu().numpy(), V, P if want_pos else 0, exact_dout, float(np.float32(scale)), drop,
                         base=_np(start) if base else None, pos_base=_np(pstart) if base else None,
                         positions=None if pos is None else pos.cpu().numpy(), seq_len=S, first=first)
    _check(gv, *t[:2], t[2] + 3, gk)
    if not base:
        assert (_np(gv)[t[2][:, 0] == 0] == 0).all()
    elif base:
        untouched = t[2][:, 0] == 0
        assert np.array_equal(_np(gv)[untouched], _np(start)[untouched])
    for w, rows, used in ((whole, V, True), (pwhole, max(P, 1), want_pos)):
        if used:
            rest = w.clone()
            rest[shift:shift + rows * (D + pad)].view(rows, -1)[:, :D] = 777.0
            assert (rest == 777.0).all(), "wrote outside its matrix"
    if want_pos:
        _check(pgv, *q[:2], q[2] + 3, gk)
    else:
        assert torch.equal(pgv.cpu(), pstart) or base == "other"
    assert layer.status() == 0
    if own:
        layer.close()
    return gv.clone(), pgv.clone()


@pytest.mark.parametrize("B,S,V,D,P,kind", CASES)
@pytest.mark.parametrize("dk,gk", list(itertools.product(T, T)))
@pytest.mark.parametrize("base", [None, "in place", "other"])
def test_gradient(ops, B, S, V, D, P, kind, dk, gk, base):
    first = P - S if kind == "run" else 0
    for index, ragged, pad, shift, p in (("i64", False, 0, 0, 0.0), ("i32", True, 8, 0, 0.1), ("i64", True, 5, 3, 0.1)):
        tok, pos = _batch(B, S, V, B + S, ragged, index, P, kind)
        _gradient(ops, tok, pos, V, D, P if kind != "none" else 0, dk, gk, first=first, base=base, pad=pad, shift=shift,
                  drop=ops.Drop(p, 8, 9) if p else None, nan_empty=ragged)


@pytest.mark.parametrize("n", [1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 511, 512, 513, 1024, 4097, 16385, 40000])
@pytest.mark.parametrize("spread", ["one token", "two tokens", "distinct", "runs", "none"])
def test_gradient_of_repeated_tokens(ops, n, spread):
    """Segments of every length, from none to all places on one token."""
    V, D = 600, 24
    rng = np.random.default_rng(n)
    tok = {"one token": np.full(n, 599), "two tokens": rng.integers(0, 2, n) * 256 + 3, "distinct": np.arange(n) % V,
           "runs": np.minimum(rng.geometric(0.02, n), V - 1), "none": np.full(n, -1)}[spread]
    tok = torch.from_numpy(tok).cuda().view(1, n)
    a = _gradient(ops, tok, None, V, D, n, "f32", "f32", drop=ops.Drop(0.2, 4, 5))
    b = _gradient(ops, tok, None, V, D, n, "f32", "f32", drop=ops.Drop(0.2, 4, 5))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), "the same call twice differs"


@pytest.mark.parametrize("n,V,share", [(16384, 50257, 0.0), (16385, 50257, 0.0), (40000, 50257, 0.1), (40000, 8, 0.0),
                                       (100000, 4000, 0.1), (131072, 50257, 0.04), (131072, 50257, 0.3), (131071, 700, 0.3),
                                       (131073, 50257, 0.1), (300000, 130000, 0.05), (2200000, 5, 0.5)])
@pytest.mark.parametrize("packed,index", [(False, torch.int64), (True, torch.int32)])
def test_sums_of_large_repeated_batches(ops, n, V, share, packed, index):
    """A share of the places holds one token and a few are empty; dout is small integers, so every sum is exact."""
    g = np.random.default_rng(n + V)
    tok = g.integers(0, V, n)
    tok[g.random(n) < share] = min(V - 1, 777)
    tok[g.random(n) < 0.01] = -1
    P = 37
    pos = g.integers(0, P, n) * (g.random(n) < 0.9)
    dout = g.integers(-2, 3, (n, 4)).astype(np.float32)
    layer = ops.TokenEmbedding(V, 4, n, positions=P)
    tables = [torch.full((rows, 4), float("nan"), device="cuda") for rows in (V, P)]
    layer.backward(torch.from_numpy(tok).to(index).cuda(), torch.from_numpy(dout).cuda(), tables[0],
                   pos_grad=tables[1] if packed else None,
                   positions=torch.from_numpy(pos).to(index).cuda() if packed else None)
    there = tok >= 0
    for got, key, rows in ((tables[0], tok, V), (tables[1], pos, P))[:2 if packed else 1]:
        want = np.stack([np.bincount(key[there], dout[there, c], rows) for c in range(4)], 1)
        assert np.array_equal(got.cpu().numpy(), want)
    assert layer.status() == 0
    layer.close()


@pytest.mark.parametrize("n", [3000, 12000, 40000, 140000])
def test_short_sums_run_in_the_places_order(ops, n):
    """Up to four places of a token are added one after the other in fp32."""
    V = 50257
    g = np.random.default_rng(n)
    tok = (g.random(n) ** 2 * V).astype(np.int64)
    dout = g.standard_normal((n, 5)).astype(np.float32)
    layer = ops.TokenEmbedding(V, 5, n)
    got = torch.empty(V, 5, device="cuda")
    layer.backward(torch.from_numpy(tok).cuda(), torch.from_numpy(dout).cuda(), got)
    want = np.zeros((V, 5), np.float32)
    np.add.at(want, tok, dout)
    few = np.bincount(tok, minlength=V) <= 4
    assert np.array_equal(got.cpu().numpy()[few], want[few])
    layer.close()


@pytest.mark.parametrize("S,P", [(1, 1), (1, 3), (2, 2), (100, 100), (7000, 7000)])
def test_position_gradient_of_many_sequences(ops, S, P):
    B = 7000 // S
    tok, _ = _batch(B, S, 300, S, True, "i64", P, "run")
    _gradient(ops, tok, None, 300, 40, P, "bf16", "f32")


@pytest.mark.parametrize("Q,S", [(32, 5), (33, 5), (64, 1), (65, 7), (129, 16), (257, 3), (1000, 9), (1024, 2), (1025, 2),
                                 (40, 3000)])
@pytest.mark.parametrize("D,dtype", [(4, torch.float32), (264, torch.bfloat16), (771, torch.bfloat16), (24, torch.float32)])
@pytest.mark.parametrize("mode", ["fresh", "in place"])
def test_running_positions_of_repeated_sequences(ops, Q, S, D, dtype, mode):
    """Positions shared by several warps: the last sequence is cut short, a few places, two whole positions and the
    whole first quarter of another are empty; dout is small integers, so every fp32 sum is exact."""
    g = np.random.default_rng(Q * S + D)
    n, P, first, V = Q * S - S // 2, S + 11, 3, 13
    tok = g.integers(0, V, n)
    tok[g.random(n) < 0.1] = -1
    spot = np.arange(n) % S
    if S > 4:
        tok[(spot == 1) | (spot == 4) | ((spot == 2) & (np.arange(n) < n // 4))] = -1
    dout = g.integers(-2, 3, (n, D)).astype(np.float32)
    base = g.integers(-3, 4, (P, D)).astype(np.float32)
    layer = ops.TokenEmbedding(V, D, n, positions=P)
    grad = torch.empty(V, D, device="cuda")
    pos_grad = torch.from_numpy(base).cuda() if mode == "in place" else torch.full((P, D), float("nan"), device="cuda")
    layer.backward(torch.from_numpy(tok).cuda(), torch.from_numpy(dout).to(dtype).cuda(), grad, pos_grad=pos_grad,
                   seq_len=S, first_position=first, pos_base=pos_grad if mode == "in place" else None)
    want = base.astype(np.float64) if mode == "in place" else np.zeros((P, D))
    there = tok >= 0
    np.add.at(want, first + spot[there], dout[there])
    assert np.array_equal(pos_grad.cpu().numpy(), want)
    assert layer.status() == 0
    layer.close()


def test_gradient_of_a_large_vocabulary(ops):
    V = 1 << 20
    tok = torch.tensor([[0, V - 1, V - 1, 1, 524288, 255, 256, 0, 131072, 77777]], device="cuda")
    layer = ops.TokenEmbedding(V, 8, 10)
    dout = _rand((10, 8), "f32", 1)
    grad = torch.full((V, 8), 9.0, device="cuda")
    layer.backward(tok, dout.cuda().view(1, 10, 8), grad)
    want = torch.zeros(V, 8, dtype=torch.float64).index_add_(0, tok.cpu().view(-1), dout.double())
    assert torch.allclose(grad.cpu().double(), want, rtol=2**-22, atol=0)
    with pytest.raises(ops.LionCubError):
        ops.TokenEmbedding(V + 1, 8, 10)


def test_empty_batch_and_reused_layer(ops):
    """A layer serves batches of any size up to its own; nothing stays from one to the next."""
    V, D, P = 300, 32, 64
    layer = ops.TokenEmbedding(V, D, 5000, positions=P, scale=1.3)
    for B, S in ((70, 64), (0, 64), (1, 1), (3, 50), (70, 64), (1, 64)):
        tok, _ = _batch(B, S, V, B, B > 1, "i64", P, "run")
        _gradient(ops, tok, None, V, D, P, "bf16", "bf16", layer=layer)
    out = layer.forward(torch.empty(0, 4, dtype=torch.int64, device="cuda"), torch.zeros(V, D, device="cuda"))
    assert out.shape == (0, 4, D)
    layer.close()
    with pytest.raises(ops.LionCubError):
        layer.forward(tok, torch.zeros(V, D, device="cuda"))


def test_gradient_against_differences(ops):
    """The lookup is linear in its tables, so a difference of the loss
    sum(out * dout) along any direction E is the gradient's product with E:
    with tables and directions on a coarse grid (multiples of 2^-6 up to 2)
    and scale 2 the fp32 lookups are exact, and so is their difference."""
    V, D, P, B, S = 90, 40, 32, 6, 32
    rng = np.random.default_rng(0)
    grid = lambda *s: torch.from_numpy(rng.integers(-128, 129, s) / 64.0).float().cuda()  # noqa: E731
    wte, wpe, e, pe, dout = grid(V, D), grid(P, D), grid(V, D), grid(P, D), grid(B, S, D)
    tok, _ = _batch(B, S, V, 3, True, "i64", P, "run")
    layer = ops.TokenEmbedding(V, D, B * S, positions=P, scale=2.0)
    drop = ops.Drop(0.5, 1, 1)  # rescaled by exactly 2
    f = lambda a, b: layer.forward(tok, a, b, drop=drop, out_dtype=torch.float32).double()  # noqa: E731
    g, pg = torch.empty(V, D, device="cuda"), torch.empty(P, D, device="cuda")
    layer.backward(tok, dout, g, pos_grad=pg, drop=drop)
    loss = ((f(wte + e, wpe + pe) - f(wte, wpe)) * dout.double()).sum().item()
    assert loss == (g.double() * e.double()).sum().item() + (pg.double() * pe.double()).sum().item()


@pytest.mark.parametrize("B,S,packed", [(3, 16, False), (200, 16, False), (3, 16, True)])
def test_rows_without_a_place_keep_their_bits(ops, B, S, packed):
    """A base row without a place, -0 and NaN included, is left (in place) or copied bit for bit: rows outside the
    batch, and positions whose places are all empty."""
    V, D, P = 50, 24, 20
    tok = torch.full((B, S), -1, dtype=torch.int64, device="cuda")
    tok[:, ::2] = 7
    pos = torch.arange(S, device="cuda").repeat(B, 1) if packed else None
    dout = torch.ones(B, S, D, device="cuda")
    layer = ops.TokenEmbedding(V, D, B * S, positions=P)
    odd = torch.tensor([-0.0, float("nan"), 0.0, float("inf")], device="cuda").repeat(6)
    base, pos_base = odd.repeat(V, 1), odd.repeat(P, 1)
    for in_place in (True, False):
        g, pg = (base.clone(), pos_base.clone()) if in_place else (torch.ones_like(base), torch.ones_like(pos_base))
        layer.backward(tok, dout, g, pos_grad=pg, base=g if in_place else base, pos_base=pg if in_place else pos_base,
                       positions=pos)
        rows = torch.arange(V) != 7
        spots = (torch.arange(P) >= S) | (torch.arange(P) % 2 == 1)
        assert torch.equal(g[rows.cuda()].view(torch.int32), base[rows.cuda()].view(torch.int32))
        assert torch.equal(pg[spots.cuda()].view(torch.int32), pos_base[spots.cuda()].view(torch.int32))
        assert (g[7, 2] == B * S // 2) and (pg[0, 2] == B)


def test_offsets_beyond_32_bits(ops):
    """Rows of a 40000 x 65536 matrix (2.6e9 elements): a lookup into it and the gradient from it, on columns of
    the last slab; every sum is a small integer, so exact."""
    n, D, V = 40000, 65536, 5
    rng = np.random.default_rng(2)
    tok = torch.from_numpy(rng.integers(0, V, n)).cuda()
    layer = ops.TokenEmbedding(V, D, n)
    table = torch.arange(V * D, device="cuda").remainder_(127).view(V, D).to(torch.bfloat16)
    x = layer.forward(tok, table)
    for lo in (0, 20000, n - 64):
        assert torch.equal(x[lo:lo + 64], table[tok[lo:lo + 64]])
    x.zero_()
    x[:, -300:] = 1.0
    x[n - 1, -1] = 3.0
    grad = torch.empty(V, D, device="cuda")
    layer.backward(tok, x, grad)
    count = torch.bincount(tok, minlength=V).float()
    want = count[:, None].repeat(1, 300)
    want[tok[n - 1], -1] += 2.0
    assert torch.equal(grad[:, -300:], want) and (grad[:, :-300] == 0).all()
    assert layer.status() == 0


def test_everything_dropped(ops):
    """p == 1: zeros, whatever the values, and gradients that only copy their base."""
    V, D, P, n = 40, 24, 8, 32
    layer = ops.TokenEmbedding(V, D, n, positions=P)
    drop = ops.Drop(1.0, 3, 4)
    tok = torch.arange(n, device="cuda").view(4, 8) % 5
    table = torch.full((V, D), float("inf"), device="cuda")
    assert (layer.forward(tok, table, table[:P], drop=drop) == 0).all()
    base, pos_base = _rand((V, D), "f32", 1).cuda(), _rand((P, D), "f32", 2).cuda()
    grad, pos_grad = torch.empty_like(base), torch.empty_like(pos_base)
    layer.backward(tok, table[:n].view(4, 8, D), grad, base=base, pos_grad=pos_grad, pos_base=pos_base, drop=drop)
    assert torch.equal(grad, base) and torch.equal(pos_grad, pos_base)


# ---- streams, graphs, layouts ------------------------------------------------------

def test_other_streams_and_graphs(ops):
    V, D, P, B, S = 500, 96, 64, 4, 64
    tok, _ = _batch(B, S, V, 1, True, "i64", P, "run")
    table, wpe = _rand((V, D), "f32", 1).cuda(), _rand((P, D), "f32", 2).cuda()
    dout = _rand((B, S, D), "bf16", 3).cuda()
    drop = ops.Drop(0.1, 6, 7)
    layer = ops.TokenEmbedding(V, D, B * S, positions=P)
    g, pg = torch.empty(V, D, device="cuda"), torch.empty(P, D, device="cuda")

    def everything(**kw):
        x = layer.forward(tok, table, wpe, drop=drop, **kw)
        layer.backward(tok, dout, g, pos_grad=pg, drop=drop, **kw)
        return x, g, pg, ops.dropout(x, drop, residual=dout, **kw), ops.dropout_backward(dout, drop, **kw)

    want = [t.clone() for t in everything()]
    g.zero_()
    pg.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = everything(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = everything()
    for t in held:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, held))
    assert layer.status() == 0


def test_gradient_into_a_flat_vector(ops):
    """Gradients land in wte's and wpe's slices of a worker's flat bf16 vector, the rest untouched."""
    import synth
    layout = synth.gpt2_layout(32, 1, vocab=77, n_ctx=16)
    d = synth.layout_total(layout)
    flat = torch.full((d,), 3.0, dtype=torch.bfloat16, device="cuda")
    (_, o1, n1, _), (_, o2, n2, _) = layout[:2]
    layer = ops.TokenEmbedding(77, 32, 16, positions=16)
    tok = torch.arange(16, device="cuda").view(1, 16)
    dout = _rand((1, 16, 32), "bf16", 1).cuda()
    layer.backward(tok, dout, flat[o1:o1 + n1].view(77, 32), pos_grad=flat[o2:o2 + n2].view(16, 32))
    assert torch.equal(flat[o1:o1 + 16 * 32].view(16, 32), dout[0]) and (flat[o1 + 16 * 32:o1 + n1] == 0).all()
    assert torch.equal(flat[o2:o2 + n2].view(16, 32), dout[0]) and (flat[o2 + n2:] == 3.0).all()


# ---- refusals ---------------------------------------------------------------------

def test_refusals(ops):
    V, D, P = 100, 16, 8
    layer = ops.TokenEmbedding(V, D, 32, positions=P)
    tok = torch.zeros(2, 8, dtype=torch.int64, device="cuda")
    table, wpe = torch.zeros(V, D, device="cuda"), torch.zeros(P, D, device="cuda")
    dout, grad = torch.zeros(2, 8, D, device="cuda"), torch.full((V, D), 4.0, device="cuda")
    err = (ValueError, ops.LionCubError)
    with pytest.raises(err):
        layer.forward(tok.cpu(), table)
    with pytest.raises(err):
        layer.forward(tok.to(torch.int16), table)
    with pytest.raises(err):
        layer.forward(tok, table[:-1])
    with pytest.raises(err):
        layer.forward(tok, table.half())
    with pytest.raises(err):
        layer.forward(tok, table.t().contiguous().t())
    with pytest.raises(err, match="type"):
        layer.forward(tok, table, wpe.bfloat16())
    with pytest.raises(err, match="positions"):
        layer.forward(tok, table, wpe, first_position=1)
    with pytest.raises(err, match="positions"):
        layer.forward(tok, table, wpe, first_position=-1)
    with pytest.raises(err):
        layer.forward(tok, table, wpe, positions=tok.to(torch.int32))
    with pytest.raises(err, match="places"):
        layer.forward(torch.zeros(33, dtype=torch.int64, device="cuda"), table)
    with pytest.raises(err, match="overlaps"):
        layer.forward(tok, table, out=table[:16])
    with pytest.raises(err):
        layer.forward(tok, table, out=torch.zeros(2, 8, D + 1, device="cuda"))
    for p in (-0.1, 1.1, float("nan")):
        with pytest.raises(err):
            layer.forward(tok, table, drop=ops.Drop(p, 1))
    with pytest.raises(err):
        layer.backward(tok, dout[:1], grad)
    with pytest.raises(err, match="type"):
        layer.backward(tok, dout, grad, base=grad.bfloat16())
    with pytest.raises(err, match="type"):
        layer.backward(tok, dout, grad, pos_grad=wpe.bfloat16())
    with pytest.raises(err, match="pos_base"):
        layer.backward(tok, dout, grad, pos_base=wpe)
    both = torch.zeros(V + 8, D, device="cuda")
    with pytest.raises(err, match="base"):
        layer.backward(tok, dout, both[:V], base=both[8:])
    with pytest.raises(err, match="overlap"):
        layer.backward(tok, dout, both[:V], pos_grad=both[V - 4:V + 4])
    with pytest.raises(err, match="overlaps"):
        layer.backward(tok, both[:16].view(2, 8, D), both[:V])
    with pytest.raises(err, match="base"):
        layer.backward(tok, dout, grad, base=both[:V], pos_grad=both[:P])
    with pytest.raises(err, match="base"):
        layer.backward(tok, dout, both[:V], pos_grad=wpe.clone(), pos_base=both[:P])
    flat = ops.TokenEmbedding(V, D, 32)
    with pytest.raises(err, match="position"):
        flat.forward(tok, table, torch.zeros(0, D, device="cuda"))
    assert (grad == 4.0).all() and layer.status() == 0
    x = torch.zeros(8, 24, device="cuda")
    drop = ops.Drop(0.1, 1)
    with pytest.raises(err):
        ops.dropout(x.cpu(), drop)
    with pytest.raises(err):
        ops.dropout(x.double(), drop)
    with pytest.raises(err):
        ops.dropout(x, drop, out=torch.zeros(8, 25, device="cuda"))
    with pytest.raises(err, match="type"):
        ops.dropout(x, drop, residual=x.bfloat16(), out=torch.zeros_like(x))
    with pytest.raises(err, match="overlaps"):
        ops.dropout(x.view(-1)[:96], drop, out=x.view(-1)[8:104])
    with pytest.raises(err, match="distance"):
        ops.dropout(torch.zeros(4, 6, 8, device="cuda")[:, 1:], drop)


def test_failed_allocation(ops, monkeypatch):
    monkeypatch.setenv("LIONCUB_FAIL_ALLOC", "1")
    with pytest.raises(ops.LionCubError, match="memory"):
        ops.TokenEmbedding(100, 16, 32)
    monkeypatch.delenv("LIONCUB_FAIL_ALLOC")
    ops.TokenEmbedding(100, 16, 32).close()


def test_failed_launch(ops, monkeypatch):
    """A launch that fails is reported, and the next call works."""
    monkeypatch.setenv("LIONCUB_FAIL_LAUNCH", "1")
    layer = ops.TokenEmbedding(100, 16, 32)
    tok = torch.zeros(4, dtype=torch.int64, device="cuda")
    table = _rand((100, 16), "f32", 1).cuda()
    with pytest.raises(ops.LionCubError, match="launch"):
        layer.forward(tok, table)
    assert torch.equal(layer.forward(tok, table, out_dtype=torch.float32), table[tok])


@pytest.mark.parametrize("k", [1, 2])
def test_failed_launch_of_a_gradient(ops, k, monkeypatch):
    """Whichever launch of a backward call fails, the next call is whole."""
    monkeypatch.setenv("LIONCUB_FAIL_LAUNCH", str(k))
    V, D, n = 300, 40, 3000
    layer = ops.TokenEmbedding(V, D, n)
    monkeypatch.delenv("LIONCUB_FAIL_LAUNCH")
    tok = torch.from_numpy(np.random.default_rng(k).integers(0, 9, n)).cuda()
    dout = _rand((n, D), "f32", k).cuda()
    grad, again = torch.empty(V, D, device="cuda"), torch.empty(V, D, device="cuda")
    with pytest.raises(ops.LionCubError, match="launch"):
        layer.backward(tok, dout, grad)
    layer.backward(tok, dout, grad)
    fresh = ops.TokenEmbedding(V, D, n)
    fresh.backward(tok, dout, again)
    assert torch.equal(grad, again)
