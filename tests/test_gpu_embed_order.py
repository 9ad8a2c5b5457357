"""The order of memory in the embedding gradient: sums that blocks hand to one
another, checked on every lane's columns and again and again.

dout is small integers, so every fp32 sum is exact in any order.
"""
import pytest

from tests.test_gpu_embed import ops  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def _integers(shape, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randint(-2, 3, shape, generator=g, device="cuda").to(dtype)


def _sums(keys, dout, rows):
    """Row sums over the places of each key (keys below 0: none), float64 on the GPU."""
    there = keys >= 0
    out = torch.zeros(rows, dout.shape[1], dtype=torch.float64, device="cuda")
    return out.index_put_((keys[there],), dout[there].double(), accumulate=True)


@pytest.mark.parametrize("n", [300, 5000, 40000, 70000])  # one block, and one, two and three levels of joining
@pytest.mark.parametrize("D", [256, 224, 512, 771])  # whole warps of columns, moved 16 bytes or an element at a time
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_joined_sums_on_every_lane(ops, n, D, dtype):
    """Long segments are cut into pieces that many blocks add; the last block to arrive joins their partials."""
    V = 9
    tok = torch.full((n,), 4, device="cuda")
    tok[n // 3:n // 3 + 40] = 2  # a second segment, and one that ends inside a piece
    tok[:7] = 0
    layer = ops.TokenEmbedding(V, D, n)
    grad = torch.empty(V, D, device="cuda")
    for seed in range(6):
        dout = _integers((n, D), dtype, seed)
        grad.fill_(float("nan"))
        layer.backward(tok, dout, grad)
        assert torch.equal(grad.double(), _sums(tok, dout, V)), seed
    assert layer.status() == 0
    layer.close()


@pytest.mark.parametrize("B,S,D", [(1, 1024, 768), (5, 300, 771), (64, 64, 256)])
@pytest.mark.parametrize("captured", [False, True])
def test_running_positions_of_inputs_just_written(ops, B, S, D, captured):
    """Each pass writes its tokens and dout on the stream right before the gradient reads them."""
    V, P, n = 500, S, B * S
    layer = ops.TokenEmbedding(V, D, n, positions=P)
    tokens = [torch.randint(-1, V, (B, S), device="cuda") for _ in range(2)]
    douts = [_integers((n, D), torch.bfloat16, seed) for seed in range(2)]
    place = torch.arange(n, device="cuda") % S
    want = [(_sums(t.view(-1), x, V), _sums(torch.where(t.view(-1) < 0, -1, place), x, P)) for t, x in zip(tokens, douts)]
    tok, dout = torch.empty_like(tokens[0]), torch.empty_like(douts[0])
    grad, pos_grad = torch.empty(V, D, device="cuda"), torch.empty(P, D, device="cuda")

    def one(k):
        grad.fill_(float("nan"))
        pos_grad.fill_(float("nan"))
        tok.copy_(tokens[k])
        dout.copy_(douts[k])
        layer.backward(tok, dout.view(B, S, D), grad, pos_grad=pos_grad)

    passes = [lambda: one(0), lambda: one(1)]
    if captured:
        one(0)
        graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
        for k, graph in enumerate(graphs):
            with torch.cuda.graph(graph):
                one(k)
        passes = [graph.replay for graph in graphs]
    for k in range(20):
        passes[k % 2]()
        got = grad.clone(), pos_grad.clone()
        assert all(torch.equal(a.double(), b) for a, b in zip(got, want[k % 2])), k
    assert layer.status() == 0
    layer.close()


def test_running_positions_after_a_call_without_its_row_sums(ops, monkeypatch):
    """A gradient whose second launch fails leaves its sort behind; the next ones, direct and replayed in turn, read
    inputs written right before them all the same."""
    B, S, D, V = 64, 64, 256, 500
    n, P = B * S, S
    monkeypatch.setenv("LIONCUB_FAIL_LAUNCH", "4")
    layer = ops.TokenEmbedding(V, D, n, positions=P)
    monkeypatch.delenv("LIONCUB_FAIL_LAUNCH")
    tokens = [torch.randint(-1, V, (B, S), device="cuda") for _ in range(2)]
    douts = [_integers((n, D), torch.float32, seed) for seed in range(2)]
    place = torch.arange(n, device="cuda") % S
    want = [(_sums(t.view(-1), x, V), _sums(torch.where(t.view(-1) < 0, -1, place), x, P)) for t, x in zip(tokens, douts)]
    tok, dout = torch.empty_like(tokens[0]), torch.empty_like(douts[0])
    grad, pos_grad = torch.empty(V, D, device="cuda"), torch.empty(P, D, device="cuda")

    def one(k, with_positions=True):
        pos_grad.fill_(float("nan"))
        tok.copy_(tokens[k])
        dout.copy_(douts[k])
        layer.backward(tok, dout.view(B, S, D), grad, pos_grad=pos_grad if with_positions else None)

    one(0)
    with pytest.raises(ops.LionCubError, match="launch"):
        one(1)
    one(0)
    assert torch.equal(grad.double(), want[0][0]) and torch.equal(pos_grad.double(), want[0][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one(1)
    for k in range(30):
        go = [lambda: one(0), graph.replay, lambda: one(0, with_positions=False)][k % 3]
        go()
        got = grad.clone(), pos_grad.clone()
        assert torch.equal(got[0].double(), want[k % 3 == 1][0]), k
        if k % 3 < 2:
            assert torch.equal(got[1].double(), want[k % 3][1]), k
    assert layer.status() == 0
    layer.close()
