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
