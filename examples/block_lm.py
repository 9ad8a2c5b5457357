"""A small transformer language model trained by the compressed Lion step, its
input layer, norms, rotary positions and gated activations by this library's
operators, with what the backward pass needs of them kept in 8 bits.

W data-parallel workers are simulated on one GPU: each has its own batch and its
own flat bf16 gradient; theta is shared.  A block is
    h = x + attention(rotary(norm(x) Wqkv)) Wo,    y = h + (silu(norm(h) Wg) * norm(h) Wu) Wd
and the head is tied to wte.  Norms keep the sum that they normed and the
activation its two inputs, as codes of 8 bits; the normed rows and the
activation's result, which the weight gradients of the products need, are
computed again from them in the backward pass.  torch computes the products,
attention's softmax and the loss.

    python examples/block_lm.py [--steps 60] [--workers 2] [--blocks 2] [--keep int8|e4m3|full]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

from communication_compressed_sign_gb300 import (
    MODE_SIGN_MAJORITY, TENSOR_SYNC_M, LionCubOptimizer, Packed, RmsNorm, Rotary, TokenEmbedding, activation, activation_backward,
)

VOCAB, WIDTH, HEADS, HIDDEN, SEQ, BATCH = 509, 128, 4, 256, 64, 8
CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn, "full": None}


def layout(blocks):
    """(name, shape) -> (shape, offset, numel, flags) of one flat vector."""
    shapes = {"wte": (VOCAB, WIDTH), "norm": (WIDTH,)}
    for b in range(blocks):
        shapes.update({f"{b}.norm1": (WIDTH,), f"{b}.qkv": (WIDTH, 3 * WIDTH), f"{b}.out": (WIDTH, WIDTH), f"{b}.norm2": (WIDTH,),
                       f"{b}.gate_up": (WIDTH, 2 * HIDDEN), f"{b}.down": (HIDDEN, WIDTH)})
    out, at = {}, 0
    for name, shape in shapes.items():
        n = torch.Size(shape).numel()
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


class Model:
    """The operators' handles, shared by all workers; a worker's step is :meth:`gradients`."""

    def __init__(self, blocks, keep="int8"):
        self.blocks, self.codes = blocks, CODES[keep]
        self.embedding = TokenEmbedding(VOCAB, WIDTH, BATCH * SEQ)
        self.norm, self.rotary = RmsNorm(WIDTH), Rotary(WIDTH // HEADS)
        self.mask = torch.full((SEQ, SEQ), float("-inf"), device="cuda").triu(1)

    def kept(self, rows, cols):
        """Room for what is kept of a matrix, or None: the matrix itself is kept."""
        return None if self.codes is None else Packed.empty((rows, cols), group=64, dtype=self.codes)

    def normed(self, x, weight, residual=None):
        """(normed rows, x + residual, what the backward pass needs)."""
        n, D = x.shape
        rstd, saved = torch.empty(n, device="cuda"), self.kept(n, D)
        h = x if residual is None else torch.empty_like(residual)
        y = self.norm.forward(x, weight, residual=residual, summed=None if residual is None else h, saved=saved, rstd=rstd)
        return y, h, (h if saved is None else saved, rstd)

    def norm_gradient(self, dy, kept, weight, grad, residual_grad=None):
        """(gradient of the sum, the normed rows again); weight's gradient is written into grad."""
        again = torch.empty_like(dy)
        dx = self.norm.backward(dy, *kept, weight, residual_grad=residual_grad, weight_grad=grad, again=again)
        return dx, again

    def gradients(self, p, g, tokens, targets):
        """One worker's loss; its gradients are written into the views g of its flat vector."""
        n, d = tokens.numel(), WIDTH // HEADS
        heads = lambda t: t.view(BATCH, SEQ, 3, HEADS, d).unbind(2)  # noqa: E731
        x = self.embedding.forward(tokens, p["wte"], out_dtype=torch.float32).view(n, WIDTH)
        tape, branch = [], None  # branch: what the last block adds to x
        for b in range(self.blocks):
            w = {k[len(f"{b}."):]: v for k, v in p.items() if k.startswith(f"{b}.")}
            y, x, kept1 = self.normed(x, w["norm1"]) if branch is None else self.normed(branch, w["norm1"], residual=x)
            q, k, v = heads(y @ w["qkv"])
            self.rotary.forward(q, k, q_out=q, k_out=k)
            probs = torch.softmax(torch.einsum("bshd,bthd->bhst", q, k) * d ** -0.5 + self.mask, -1)
            o = torch.einsum("bhst,bthd->bshd", probs, v).reshape(n, WIDTH)
            y, x, kept2 = self.normed(o @ w["out"], w["norm2"], residual=x)
            both = y @ w["gate_up"]
            gate, up = both[:, :HIDDEN], both[:, HIDDEN:]
            packs = self.kept(n, HIDDEN), self.kept(n, HIDDEN)
            a = activation(gate, up, kind="silu", saved=packs[0], saved_up=packs[1])
            branch = a @ w["down"]
            tape.append((w, kept1, q, k, v, probs, o, kept2, (gate, up) if packs[0] is None else packs))
        y, x, kept = self.normed(branch, p["norm"], residual=x)
        logits = y @ p["wte"].t()
        loss = torch.nn.functional.cross_entropy(logits, targets.reshape(-1))

        dlogits = torch.softmax(logits, 1)
        dlogits[torch.arange(n, device="cuda"), targets.reshape(-1)] -= 1
        dlogits /= n
        dx, again = self.norm_gradient(dlogits @ p["wte"], kept, p["norm"], g["norm"])
        head = (dlogits.t() @ again).to(g["wte"].dtype)
        for b in reversed(range(self.blocks)):
            w, kept1, q, k, v, probs, o, kept2, (gate, up) = tape[b]
            a, dboth = torch.empty(n, HIDDEN, device="cuda"), torch.empty(n, 2 * HIDDEN, device="cuda")
            activation_backward(dx @ w["down"].t(), gate, up, kind="silu", dx=dboth[:, :HIDDEN], dup=dboth[:, HIDDEN:], again=a)
            g[f"{b}.down"].copy_(a.t() @ dx)
            dx, again = self.norm_gradient(dboth @ w["gate_up"].t(), kept2, w["norm2"], g[f"{b}.norm2"], residual_grad=dx)
            g[f"{b}.gate_up"].copy_(again.t() @ dboth)
            g[f"{b}.out"].copy_(o.t() @ dx)
            do = (dx @ w["out"].t()).view(BATCH, SEQ, HEADS, d)
            dqkv = torch.empty(n, 3 * WIDTH, device="cuda")
            dq, dk, dv = heads(dqkv)
            dv.copy_(torch.einsum("bhst,bshd->bthd", probs, do))
            dp = torch.einsum("bshd,bthd->bhst", do, v)
            ds = probs * (dp - (dp * probs).sum(-1, keepdim=True)) * d ** -0.5
            dq.copy_(torch.einsum("bhst,bthd->bshd", ds, k))
            dk.copy_(torch.einsum("bhst,bshd->bthd", ds, q))
            self.rotary.backward(dq, dk, q_out=dq, k_out=dk)
            dx, again = self.norm_gradient(dqkv @ w["qkv"].t(), kept1, w["norm1"], g[f"{b}.norm1"], residual_grad=dx)
            g[f"{b}.qkv"].copy_(again.t() @ dqkv)
        self.embedding.backward(tokens, dx.view(*tokens.shape, WIDTH), g["wte"], base=head)
        return loss

    def close(self):
        assert self.embedding.status() == 0 and self.norm.status() == 0
        for h in (self.embedding, self.norm, self.rotary):
            h.close()


def initial(table, d, generator):
    theta = torch.randn(d, generator=generator, device="cuda") * 0.05
    for name, (_, at, n, _) in table.items():
        if "norm" in name:
            theta[at:at + n] = 1.0
    return theta


def train(steps=60, workers=2, blocks=2, keep="int8", seed=0, log=print):
    table, d = layout(blocks)
    generator = torch.Generator(device="cuda")
    generator.manual_seed(seed)
    theta = initial(table, d, generator)
    momenta = [torch.zeros(d, device="cuda") for _ in range(workers)]
    grads = [torch.empty(d, dtype=torch.bfloat16, device="cuda") for _ in range(workers)]
    params, slots = views(theta, table), [views(g, table) for g in grads]
    opt = LionCubOptimizer(d, workers, [(at, n, flags) for _, at, n, flags in table.values()], lr=1e-3, wd=0.01,
                           mode=MODE_SIGN_MAJORITY, nbits=1, sync_interval=10)
    opt.bind(theta, momenta)
    model, losses = Model(blocks, keep), []
    for step in range(steps):
        total = 0.0
        for w in range(workers):
            t = sequences(BATCH, generator)
            total = total + model.gradients(params, slots[w], t[:, :-1].contiguous(), t[:, 1:].contiguous())
        opt.step(grads)
        losses.append(float(total) / workers)
        if log and (step % 10 == 0 or step == steps - 1):
            log(f"step {step:4d}  loss {losses[-1]:.3f}")
    model.close()
    opt.close()
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--workers", type=int, default=2)
    ap.add_argument("--blocks", type=int, default=2)
    ap.add_argument("--keep", choices=list(CODES), default="int8", help="how norms and activations keep what their backward pass needs")
    args = ap.parse_args()
    train(args.steps, args.workers, args.blocks, args.keep)
