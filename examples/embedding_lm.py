"""A small language model trained by the compressed Lion step, its input layer
and dropout by this library's operators.

W data-parallel workers are simulated on one GPU, as the library does: each has
its own batch, its own dropout streams and its own flat bf16 gradient; theta is
shared.  The model is an input layer drop(wte[token] + wpe[position]), one
residual block x + drop(tanh(x W1) W2) and a head tied to wte.  The head's
gradient of wte comes first; the lookup's is added to it as the base while the
gradient is laid into the worker's flat vector, whose wte is the tensor with
synchronized momentum.  torch computes the matrix products and the loss.

    python examples/embedding_lm.py [--steps 60] [--workers 4] [--l1]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

from communication_compressed_sign_gb300 import (
    MODE_L1_INTSUM, MODE_SIGN_MAJORITY, TENSOR_SYNC_M, Drop, LionCubOptimizer, TokenEmbedding, dropout, dropout_backward,
)

VOCAB, WIDTH, SEQ, BATCH = 509, 128, 64, 16
SITES = 2  # dropout sites: the input layer and the block


def layout():
    """(name, shape) -> (offset, numel, flags) of one flat vector."""
    shapes = {"wte": (VOCAB, WIDTH), "wpe": (SEQ, WIDTH), "w1": (WIDTH, 4 * WIDTH), "w2": (4 * WIDTH, WIDTH)}
    out, at = {}, 0
    for name, shape in shapes.items():
        n = shape[0] * shape[1]
        out[name] = (shape, at, n, TENSOR_SYNC_M if name == "wte" else 0)
        at += n
    return out, at


def views(flat, table):
    return {name: flat[at:at + n].view(shape) for name, (shape, at, n, _) in table.items()}


def sequences(count, generator):
    """Tokens that mostly follow a fixed rule (next = 3 t + 7), so that there is something to learn."""
    t = torch.randint(0, VOCAB, (count,), generator=generator, device="cuda")
    out = [t]
    for _ in range(SEQ):
        jump = torch.rand(count, generator=generator, device="cuda") < 0.1
        t = torch.where(jump, torch.randint(0, VOCAB, (count,), generator=generator, device="cuda"), (3 * t + 7) % VOCAB)
        out.append(t)
    return torch.stack(out, 1)


def gradients(layer, p, g, tokens, targets, p_drop, seed, stream):
    """One worker's loss; its gradients are written into the views g of its flat vector."""
    n = tokens.numel()
    first, second = Drop(p_drop, seed, stream), Drop(p_drop, seed, stream + 1)
    x = layer.forward(tokens, p["wte"], p["wpe"], drop=first, out_dtype=torch.float32).view(n, WIDTH)
    a = torch.tanh(x @ p["w1"])
    h = dropout(a @ p["w2"], second, residual=x)
    logits = h @ p["wte"].t()
    loss = torch.nn.functional.cross_entropy(logits, targets.reshape(-1))

    dlogits = torch.softmax(logits, 1)
    dlogits[torch.arange(n, device="cuda"), targets.reshape(-1)] -= 1
    dlogits /= n
    head = (dlogits.t() @ h).to(torch.bfloat16)
    dh = dlogits @ p["wte"]
    dm = dropout_backward(dh, second)
    g["w2"].copy_(a.t() @ dm)
    da = (dm @ p["w2"].t()) * (1 - a * a)
    g["w1"].copy_(x.t() @ da)
    dx = dh + da @ p["w1"].t()
    layer.backward(tokens, dx.view(*tokens.shape, WIDTH), g["wte"], base=head, pos_grad=g["wpe"], drop=first)
    return loss


def train(steps=60, workers=4, l1=False, p_drop=0.1, seed=0, log=print):
    table, d = layout()
    generator = torch.Generator(device="cuda")
    generator.manual_seed(seed)
    theta = torch.randn(d, generator=generator, device="cuda") * 0.05
    momenta = [torch.zeros(d, device="cuda") for _ in range(workers)]
    grads = [torch.empty(d, dtype=torch.bfloat16, device="cuda") for _ in range(workers)]
    params, slots = views(theta, table), [views(g, table) for g in grads]
    opt = LionCubOptimizer(d, workers, [(at, n, flags) for _, at, n, flags in table.values()], lr=1e-3, wd=0.01,
                           mode=MODE_L1_INTSUM if l1 else MODE_SIGN_MAJORITY, nbits=4 if l1 else 1, sync_interval=10)
    opt.bind(theta, momenta)
    layer = TokenEmbedding(VOCAB, WIDTH, BATCH * SEQ, positions=SEQ)
    losses = []
    for step in range(steps):
        total = 0.0
        for w in range(workers):
            t = sequences(BATCH, generator)
            total = total + gradients(layer, params, slots[w], t[:, :-1].contiguous(), t[:, 1:].contiguous(), p_drop, seed,
                                      (step * workers + w) * SITES)
        opt.step(grads)
        losses.append(float(total) / workers)
        if log and (step % 10 == 0 or step == steps - 1):
            log(f"step {step:4d}  loss {losses[-1]:.3f}")
    assert layer.status() == 0
    layer.close()
    opt.close()
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--workers", type=int, default=4)
    ap.add_argument("--l1", action="store_true", help="4-bit L1 codes instead of signs")
    args = ap.parse_args()
    train(args.steps, args.workers, args.l1)
