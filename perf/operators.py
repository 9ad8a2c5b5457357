"""What is measured of the input-layer operators: the embedding lookup, its
gradient by sorted tokens, and dropout from a counter-based generator.

A GPT-2 style input layer is drop(scale * wte[token] + wpe[position]); its
gradient fills the first two tensors of the flat vector that a compressed Lion
step reads.  Where ``own`` is false, :func:`run` computes the same with
elementary torch operations.  Sizes come from the layouts in ``synth``
(vocabulary 50257, 1024 positions; widths 192, 768, 1024, 2048).
"""
import math

import numpy as np
import torch

own = False

VOCAB, POSITIONS = 50257, 1024
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "bf16": 2, "i32": 4, "i64": 8}


def _lookup(name, batch, seq, dim, **more):
    c = dict(name=name, op="lookup", batch=batch, seq=seq, vocab=VOCAB, dim=dim, table="f32", out="bf16", index="i64",
             pos="run", first=0, p=0.0, ragged=False, scale=1.0)
    return {**c, **more}


def _grad(name, batch, seq, dim, **more):
    c = dict(name=name, op="grad", batch=batch, seq=seq, vocab=VOCAB, dim=dim, dout="bf16", grad="bf16", index="i64",
             pos="none", p=0.0, ragged=False, scale=1.0, base=False)
    return {**c, **more}


def _dropout(name, rows, cols, **more):
    c = dict(name=name, op="dropout", rows=rows, cols=cols, x="bf16", out="bf16", residual=False, backward=False,
             pad=0, p=0.1)
    return {**c, **more}


def listed():
    return [
        # one new token for each of 8 sequences that are being answered (GPT-2 small, fp32 parameters): latency
        _lookup("lookup-decode", 8, 1, 768, first=511),
        # a worker's batch of 8 full sequences in training
        _lookup("lookup-train", 8, 1024, 768, p=0.1),
        # the widest layout, 64 sequences at once
        _lookup("lookup-large", 64, 1024, 2048, p=0.1),
        # a small vocabulary and an odd width, sequences packed one after the other, the last places empty
        _lookup("lookup-odd", 7, 701, 771, vocab=1003, table="bf16", out="f32", index="i32", pos="packed", ragged=True,
                scale=27.75),
        # one sequence a worker: the dense gradient of wte, nearly all of it zero rows, and of wpe
        _grad("grad-one-sequence", 1, 1024, 768, pos="run", p=0.1),
        # an ordinary batch, GPT-2 medium, no dropout
        _grad("grad-train", 16, 1024, 1024),
        # tied embeddings: the head's gradient is there already and the lookup's is added to it
        _grad("grad-tied", 16, 1024, 768, base=True, p=0.1),
        # the largest batch of the widest layout, both tables
        _grad("grad-large", 64, 1024, 2048, pos="run", p=0.1),
        # fp32 gradients of a small vocabulary and an odd width, packed sequences with empty places
        _grad("grad-odd", 29, 701, 771, vocab=1003, dout="f32", grad="f32", index="i32", pos="packed", ragged=True,
              scale=27.75, p=0.25),
        # DeiT-Tiny's tokens (197 of width 192) of a few images, fp32
        _dropout("dropout-small", 4 * 197, 192, x="f32", out="f32"),
        # a block's output joins the residual stream: GPT-2 small, 8 sequences
        _dropout("dropout-residual", 8192, 768, out="f32", residual=True),
        # its gradient at the widest layout
        _dropout("dropout-back-large", 65536, 2048, backward=True),
    ]


def _log_int(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _width(rng):
    d = _log_int(rng, 64, 2048)
    return d if rng.random() < 0.3 else max(64, d // 64 * 64)


def draw(rng):
    top = {c["op"]: max(work(k)["bytes"] for k in listed() if k["op"] == c["op"]) for c in listed()}
    while True:
        op = rng.choice(["lookup", "grad", "grad", "dropout"])
        kind = lambda: "bf16" if rng.random() < 0.7 else "f32"  # noqa: E731
        if op == "dropout":
            c = _dropout(None, _log_int(rng, 8, 65536), _width(rng), x=kind(), out=kind(), residual=rng.random() < 0.4,
                         backward=rng.random() < 0.4, pad=rng.choice([0, 0, 0, 64, 5]), p=rng.choice([0.1, 0.1, 0.3]))
            c["residual"] = c["residual"] and not c["backward"]
        else:
            seq = _log_int(rng, 1, POSITIONS) if rng.random() < 0.5 else POSITIONS
            vocab = VOCAB if rng.random() < 0.6 else _log_int(rng, 256, VOCAB)
            more = dict(vocab=vocab, index=rng.choice(["i64", "i64", "i32"]), pos=rng.choice(["none", "run", "packed"]),
                        ragged=rng.random() < 0.3, p=rng.choice([0.0, 0.1, 0.1, 0.2]), scale=rng.choice([1.0, 1.0, 22.5]))
            if op == "lookup":
                first = rng.randrange(0, POSITIONS - seq + 1) if more["pos"] == "run" else 0
                c = _lookup(None, _log_int(rng, 1, 64), seq, _width(rng), first=first, **{**more, "table": kind(), "out": kind()})
            else:
                t = kind()
                c = _grad(None, _log_int(rng, 1, 64), seq, _width(rng), **{**more, "dout": kind(), "grad": t,
                                                                           "base": rng.random() < 0.25})
        c.pop("name")
        if work(c)["bytes"] <= top[op]:
            return c


# ---- inputs ------------------------------------------------------------------

def _weights(vocab):
    """Relative frequency of token ids: by rank, as a subword vocabulary has them."""
    return 1.0 / (np.arange(vocab, dtype=np.float64) + 2.7)


def _batch(case, g):
    """Token ids (batch * seq), -1 at the empty places, and their positions (None: first + place in the sequence)."""
    dev, B, S = "cuda", case["batch"], case["seq"]
    cdf = torch.from_numpy(np.cumsum(_weights(case["vocab"]))).to(dev)
    u = torch.rand(B * S, generator=g, device=dev, dtype=torch.float64) * cdf[-1]
    tokens = torch.searchsorted(cdf, u, right=True).clamp_(max=case["vocab"] - 1)
    place = torch.arange(B * S, device=dev) % S
    if case["ragged"]:  # each sequence has a length of its own, half of S at least
        length = torch.randint((S + 1) // 2, S + 1, (B,), generator=g, device=dev)
        tokens = torch.where(place < length.repeat_interleave(S), tokens, torch.full_like(tokens, -1))
    positions = None
    if case["pos"] == "packed":  # documents end at random, and the next one begins at position 0
        begins = (torch.rand(B * S, generator=g, device=dev) < 4.0 / S) | (place == 0)
        at = torch.where(begins, place, torch.zeros_like(place)).view(B, S).cummax(1).values.view(-1)
        positions = place - at
    to = torch.int32 if case["index"] == "i32" else torch.int64
    return tokens.to(to).view(B, S), None if positions is None else positions.to(to).view(B, S)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 17)

    def normal(rows, cols, kind, std, width=None):
        x = torch.randn(rows, width or cols, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(TYPES[kind])
        return x[:, :cols]

    s = {"case": case, "seed": 7919 * seed + 5, "stream": seed % 1000}
    if case["op"] == "dropout":
        s["x"] = normal(case["rows"], case["cols"], case["x"], 1.0, case["cols"] + case["pad"])
        if case["residual"]:
            s["residual"] = normal(case["rows"], case["cols"], case["out"], 1.0)
        s["result"] = torch.empty(case["rows"], case["cols"], dtype=TYPES[case["out"]], device="cuda")
        return s
    V, D = case["vocab"], case["dim"]
    s["tokens"], s["positions"] = _batch(case, g)
    n = s["tokens"].numel()
    if case["op"] == "lookup":
        s["wte"] = normal(V, D, case["table"], 0.02)
        s["wpe"] = normal(POSITIONS, D, case["table"], 0.01) if case["pos"] != "none" else None
        s["result"] = torch.empty(case["batch"], case["seq"], D, dtype=TYPES[case["out"]], device="cuda")
    else:
        s["dout"] = normal(n, D, case["dout"], 1e-3).view(case["batch"], case["seq"], D)
        s["base"] = normal(V, D, case["grad"], 1e-3) if case["base"] else None
        s["grad"] = torch.empty(V, D, dtype=TYPES[case["grad"]], device="cuda")
        s["pos_grad"] = torch.empty(POSITIONS, D, dtype=TYPES[case["grad"]], device="cuda") if case["pos"] != "none" else None
    if own:
        from communication_compressed_sign_gb300 import TokenEmbedding
        s["layer"] = TokenEmbedding(V, D, n, positions=POSITIONS if case["pos"] != "none" else 0, scale=case["scale"])
    return s


# ---- one pass ------------------------------------------------------------------

def _threshold(p):
    return int(math.floor(p * 65536 + 0.5))


def _rescale(p):
    """1 / (the share that is kept), in fp32."""
    return float(np.float32(65536.0 / (65536 - _threshold(p))))


def _signed(x):
    x &= (1 << 64) - 1
    return x - (1 << 64) if x >> 63 else x


def _shift(z, by):
    return (z >> by) & ((1 << (64 - by)) - 1)


def _mixed(z):
    z = (z ^ _shift(z, 30)) * _signed(0xbf58476d1ce4e5b9)
    z = (z ^ _shift(z, 27)) * _signed(0x94d049bb133111eb)
    return z ^ _shift(z, 31)


def _keep(shape, p, seed, stream):
    """Which elements stay: element e, row by row, has the 16-bit field e % 4 of output e // 4 of the generator that
    starts from output `stream` of the one that starts from `seed`."""
    n = int(np.prod(shape))
    step = _signed(0x9e3779b97f4a7c15)
    key = _mixed(torch.tensor([_signed(seed + (stream + 1) * 0x9e3779b97f4a7c15)], device="cuda"))
    z = _mixed(key + torch.arange(1, (n + 3) // 4 + 1, device="cuda") * step)
    field = z.view(torch.int16).to(torch.int32) & 0xffff
    return (field[:n] >= _threshold(p)).view(shape)


def _plain_lookup(s, case):
    D = case["dim"]
    tokens = s["tokens"].reshape(-1).long()
    there = tokens >= 0
    y = s["wte"][tokens.clamp(min=0)].float() * case["scale"]
    if case["pos"] != "none":
        y = y + s["wpe"][_positions(s, case)].float()
    y = torch.where(there[:, None], y, torch.zeros_like(y))
    if case["p"]:
        y = torch.where(_keep(y.shape, case["p"], s["seed"], s["stream"]), y * _rescale(case["p"]), torch.zeros_like(y))
    return y.to(TYPES[case["out"]]).view(case["batch"], case["seq"], D)


def _positions(s, case):
    if s["positions"] is not None:
        return s["positions"].reshape(-1).long()
    return torch.arange(case["batch"] * case["seq"], device="cuda") % case["seq"] + case.get("first", 0)


def _plain_grad(s, case):
    V, D = case["vocab"], case["dim"]
    tokens = s["tokens"].reshape(-1).long()
    x = s["dout"].reshape(-1, D).float()
    keep, r = (tokens >= 0)[:, None], 1.0
    if case["p"]:
        keep, r = keep & _keep(x.shape, case["p"], s["seed"], s["stream"]), _rescale(case["p"])
    x = torch.where(keep, x, torch.zeros_like(x))
    dw = torch.zeros(V, D, device="cuda").index_add_(0, tokens.clamp(min=0), x) * (case["scale"] * r)
    if case["base"]:
        dw = dw + s["base"].float()
    dw = dw.to(TYPES[case["grad"]])
    if case["pos"] == "none":
        return {"wte": dw}
    dp = torch.zeros(POSITIONS, D, device="cuda").index_add_(0, _positions(s, case), x) * r
    return {"wte": dw, "wpe": dp.to(TYPES[case["grad"]])}


def _plain_dropout(s, case):
    x = s["x"].float()
    y = torch.where(_keep(x.shape, case["p"], s["seed"], s["stream"]), x * _rescale(case["p"]), torch.zeros_like(x))
    if case["residual"]:
        y = y + s["residual"].float()
    return y.to(TYPES[case["out"]])


def run(state):
    s, case = state, state["case"]
    if not own:
        return {"lookup": _plain_lookup, "grad": _plain_grad, "dropout": _plain_dropout}[case["op"]](s, case)
    from communication_compressed_sign_gb300 import Drop, dropout, dropout_backward
    drop = Drop(case["p"], s["seed"], s["stream"]) if case["p"] else None
    if case["op"] == "lookup":
        return s["layer"].forward(s["tokens"], s["wte"], s["wpe"], positions=s["positions"], first_position=case["first"],
                                  drop=drop, out=s["result"])
    if case["op"] == "grad":
        s["layer"].backward(s["tokens"], s["dout"], s["grad"], pos_grad=s["pos_grad"], positions=s["positions"],
                            base=s["base"], drop=drop)
        return {"wte": s["grad"]} if s["pos_grad"] is None else {"wte": s["grad"], "wpe": s["pos_grad"]}
    if case["backward"]:
        return dropout_backward(s["x"], drop, out=s["result"])
    return dropout(s["x"], drop, residual=s.get("residual"), out=s["result"])


# ---- what a pass cannot do without ----------------------------------------------

def work(case):
    if case["op"] == "dropout":
        n = case["rows"] * case["cols"]
        each = SIZES[case["x"]] + SIZES[case["out"]] * (2 if case["residual"] else 1)
        return {"bytes": n * each, "flops": n * (2 if case["residual"] else 1)}
    n, D, V = case["batch"] * case["seq"], case["dim"], case["vocab"]
    there = n * (0.75 if case["ragged"] else 1.0)
    byte = n * SIZES[case["index"]] * (2 if case["pos"] == "packed" else 1)
    if case["op"] == "lookup":
        w = _weights(V)
        rows = float(np.sum(-np.expm1(there * np.log1p(-w / w.sum()))))  # distinct tokens that are to be expected
        byte += rows * D * SIZES[case["table"]] + n * D * SIZES[case["out"]]
        if case["pos"] != "none":
            byte += case["seq"] * D * SIZES[case["table"]]
        return {"bytes": byte, "flops": there * D * ((case["pos"] != "none") + 1 + (case["p"] > 0))}
    byte += there * D * SIZES[case["dout"]] + V * D * SIZES[case["grad"]] * (2 if case["base"] else 1)
    if case["pos"] != "none":
        byte += POSITIONS * D * SIZES[case["grad"]]
    return {"bytes": byte, "flops": there * D * (2 if case["pos"] != "none" else 1) + V * D}


# ---- the definition in 64 bits ---------------------------------------------------

def _kept_exact(rows, cols, p, seed, stream):
    """The mask again, with numpy's unsigned 64-bit numbers."""
    m1, m2, m3 = (np.uint64(v) for v in (0x9e3779b97f4a7c15, 0xbf58476d1ce4e5b9, 0x94d049bb133111eb))

    def output(start, k):
        with np.errstate(over="ignore"):
            z = np.uint64(start) + (k + np.uint64(1)) * m1
            z ^= z >> np.uint64(30)
            z *= m2
            z ^= z >> np.uint64(27)
            z *= m3
            z ^= z >> np.uint64(31)
        return z

    n = rows * cols
    key = output(seed, np.array([stream], dtype=np.uint64))[0]
    z = output(key, np.arange((n + 3) // 4, dtype=np.uint64))
    fields = np.ascontiguousarray(z.astype("<u8", copy=False)).view("<u2")[:n]
    limit = np.floor(np.float64(p) * 65536 + 0.5)
    return torch.from_numpy(fields >= limit).to("cuda").view(rows, cols), 65536.0 / (65536.0 - float(limit))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "dropout":
        keep, r = _kept_exact(case["rows"], case["cols"], case["p"], s["seed"], s["stream"])
        y = s["x"].double().masked_fill(~keep, 0.0) * r
        return y + s["residual"].double() if case["residual"] else y
    B, S, D, V = case["batch"], case["seq"], case["dim"], case["vocab"]
    n = B * S
    tokens = s["tokens"].reshape(n).to(torch.int64)
    empty = tokens < 0
    if case["p"]:
        keep, r = _kept_exact(n, D, case["p"], s["seed"], s["stream"])
    else:
        keep, r = None, 1.0
    if s["positions"] is not None:
        pos = s["positions"].reshape(n).to(torch.int64)
    else:
        pos = (torch.arange(S, device="cuda") + case.get("first", 0)).repeat(B)
    if case["op"] == "lookup":
        y = torch.index_select(s["wte"].double(), 0, tokens.masked_fill(empty, 0)).mul_(case["scale"])
        if case["pos"] != "none":
            y += torch.index_select(s["wpe"].double(), 0, pos)
        y[empty] = 0.0
        if keep is not None:
            y.mul_(r).masked_fill_(~keep, 0.0)
        return y.view(B, S, D)
    x = s["dout"].reshape(n, D).double()
    if keep is not None:
        x.mul_(r).masked_fill_(~keep, 0.0)
    x, pos, tokens = x[~empty], pos[~empty], tokens[~empty]
    dw = s["base"].double() if case["base"] else torch.zeros(V, D, dtype=torch.float64, device="cuda")
    dw = dw.index_put((tokens,), x * case["scale"], accumulate=True)
    if case["pos"] == "none":
        return {"wte": dw}
    dp = torch.zeros(POSITIONS, D, dtype=torch.float64, device="cuda").index_put((pos,), x, accumulate=True)
    return {"wte": dw, "wpe": dp}
