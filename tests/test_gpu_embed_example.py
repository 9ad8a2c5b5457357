"""The example that trains a small model with the input-layer operators and the
compressed step: one worker's gradients against torch's autograd, and a loss
that falls under both compressions."""
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
    import embedding_lm
    return embedding_lm


def test_gradients_equal_autograd(lm):
    """float64 autograd of the same model with the same masks; bf16 gradients
    hold 8 bits, the head's is rounded once more before the lookup's is added,
    and fp32 products lose little beside that."""
    from communication_compressed_sign_gb300 import Drop, TokenEmbedding, dropout
    table, d = lm.layout()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    theta = torch.randn(d, generator=gen, device="cuda") * 0.05
    flat = torch.full((d,), float("nan"), dtype=torch.bfloat16, device="cuda")
    t = lm.sequences(lm.BATCH, gen)
    tokens, targets = t[:, :-1].contiguous(), t[:, 1:].contiguous()
    layer = TokenEmbedding(lm.VOCAB, lm.WIDTH, tokens.numel(), positions=lm.SEQ)
    allowed = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    try:
        loss = lm.gradients(layer, lm.views(theta, table), lm.views(flat, table), tokens, targets, 0.1, 3, 40)
    finally:
        torch.backends.cuda.matmul.allow_tf32 = allowed
    n = tokens.numel()
    masks = [dropout(torch.ones(n, lm.WIDTH, device="cuda"), Drop(0.1, 3, s)).double() for s in (40, 41)]
    leaf = theta.double().requires_grad_()
    p = lm.views(leaf, table)
    x = (p["wte"][tokens] + p["wpe"][None]).view(n, -1) * masks[0]
    h = x + (torch.tanh(x @ p["w1"]) @ p["w2"]) * masks[1]
    want = torch.nn.functional.cross_entropy(h @ p["wte"].t(), targets.view(-1))
    want.backward()
    assert abs(loss.item() - want.item()) < 1e-5 * want.item()
    for name, (_, at, count, _) in table.items():
        a, b = flat[at:at + count].double(), leaf.grad[at:at + count]
        assert torch.isfinite(a).all()
        assert (a - b).norm() < 2 * 2.0**-8 * b.norm(), name


@pytest.mark.parametrize("l1", [False, True])
def test_loss_falls(lm, l1):
    losses = lm.train(steps=60, workers=4, l1=l1, log=None)
    assert losses[-1] < losses[0] - 1.0, losses[::10]
