"""The example that trains a small transformer with the block operators: it runs,
and one worker's gradients equal torch's autograd in 64 bits."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lm():
    import __graft_entry__
    __graft_entry__.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import block_lm
    return block_lm


def autograd(lm, theta, table, blocks, tokens, targets, frequencies):
    leaf = theta.double().requires_grad_()
    p = lm.views(leaf, table)
    n, d = tokens.numel(), lm.WIDTH // lm.HEADS
    norm = lambda x, w: x * (x.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * w  # noqa: E731
    angle = torch.arange(lm.SEQ, dtype=torch.float64, device="cuda")[:, None] * torch.tensor(frequencies, dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]

    def rotated(t):
        z = torch.complex(t[..., :d // 2].contiguous(), t[..., d // 2:].contiguous()) * turn
        return torch.cat([z.real, z.imag], -1)

    x = p["wte"][tokens].view(n, -1)
    mask = torch.ones(lm.SEQ, lm.SEQ, dtype=torch.bool, device="cuda").triu(1)
    for b in range(blocks):
        w = lambda name: p[f"{b}.{name}"]  # noqa: E731, B023
        q, k, v = (norm(x, w("norm1")) @ w("qkv")).view(lm.BATCH, lm.SEQ, 3, lm.HEADS, d).unbind(2)
        s = (torch.einsum("bshd,bthd->bhst", rotated(q), rotated(k)) * d ** -0.5).masked_fill(mask, float("-inf"))
        x = x + torch.einsum("bhst,bthd->bshd", torch.softmax(s, -1), v).reshape(n, -1) @ w("out")
        gate, up = (norm(x, w("norm2")) @ w("gate_up")).chunk(2, 1)
        x = x + (gate * torch.sigmoid(gate) * up) @ w("down")
    loss = torch.nn.functional.cross_entropy(norm(x, p["norm"]) @ p["wte"].t(), targets.reshape(-1))
    loss.backward()
    return loss.item(), leaf.grad


@pytest.mark.parametrize("keep", ["full", "int8", "e4m3"])
def test_gradients_equal_autograd(lm, keep):
    """bf16 gradients are off by up to 2^-9 of each number, the head's once more; fp32 products lose little beside that.
    8 bits: whole numbers are off by up to 1/254 of their group's largest, evenly spread, so 1/440 of it in the mean
    square; the largest of 64 is about 2.6 times the typical one, so 0.6 % of that.  e4m3 is off by up to 2^-4 of
    itself, 2.7 % in the mean square.  A term of a gradient has three such factors at most: 2 % and 8 %."""
    blocks = 2
    table, d = lm.layout(blocks)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    theta = lm.initial(table, d, gen)
    flat = torch.full((d,), float("nan"), dtype=torch.bfloat16, device="cuda")
    t = lm.sequences(lm.BATCH, gen)
    tokens, targets = t[:, :-1].contiguous(), t[:, 1:].contiguous()
    model = lm.Model(blocks, keep)
    allowed = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    try:
        loss = model.gradients(lm.views(theta, table), lm.views(flat, table), tokens, targets)
    finally:
        torch.backends.cuda.matmul.allow_tf32 = allowed
    want, grad = autograd(lm, theta, table, blocks, tokens, targets, model.rotary.frequencies)
    assert abs(loss.item() - want) < 1e-5 * want  # the forward pass loses nothing
    worst = {"full": 2 * 2.0 ** -8, "int8": 0.02, "e4m3": 0.08}[keep]
    for name, (_, at, count, _) in table.items():
        a, b = flat[at:at + count].double(), grad[at:at + count]
        assert torch.isfinite(a).all()
        assert (a - b).norm() < worst * b.norm(), (name, float((a - b).norm() / b.norm()))
    model.close()


def test_runs(lm):
    losses = lm.train(steps=3, workers=2, log=None)
    assert len(losses) == 3 and all(loss == loss and loss < 10 for loss in losses)
