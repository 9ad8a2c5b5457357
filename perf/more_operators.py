"""What is measured of the block operators: the root-mean-square norm with the
residual's addition and its gradient, activation checkpoints in 8 bits, the
activation whose backward pass reads them, and rotary positions.

They stand between the input layer and the matrix products of a transformer
block.  Where ``own`` is false, :func:`run` computes the same with elementary
torch operations.  Widths come from the layouts in ``synth`` (192, 768, 1024,
2048, and four times that inside a block), heads are 64 or 128 wide.

Codes of 8 bits are returned as torch's 8-bit floats beside their scales, or
restored by the operator that reads them.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}
SIZES = {"f32": 4, "bf16": 2, "int8": 1, "e4m3": 1, "i32": 4, "i64": 8, "none": 0}
TOPS = {"int8": 127.0, "e4m3": 448.0}


def _norm(name, rows, dim, **more):
    c = dict(name=name, op="norm", rows=rows, dim=dim, x="bf16", residual="bf16", out="bf16", weight="f32", group=128, pad=0)
    return {**c, **more}


def _normback(name, rows, dim, **more):
    c = dict(name=name, op="normback", rows=rows, dim=dim, dout="bf16", h="bf16", group=128, residual=True, dx="bf16",
             weight="f32", again=False, pad=0)
    return {**c, **more}


def _checkpoint(name, rows, dim, **more):
    c = dict(name=name, op="checkpoint", rows=rows, dim=dim, x="bf16", out="bf16", code="int8", group=128, pad=0)
    return {**c, **more}


def _act(name, rows, dim, **more):
    c = dict(name=name, op="act", rows=rows, dim=dim, x="bf16", kind="gelu", gated=False, code="int8", group=128, fused=False)
    return {**c, **more}


def _rotary(name, batch, seq, heads, **more):
    c = dict(name=name, op="rotary", batch=batch, seq=seq, heads=heads, kv_heads=heads, head_dim=64, rotary_dim=64, x="bf16",
             interleaved=False, index="none", first=0, scaling="none", inverse=False, fused=False)
    return {**c, **more}


def listed():
    return [
        # one new token for each of 8 sequences (GPT-2 small), the residual stream in fp32: latency
        _norm("norm-decode", 8, 768, residual="f32"),
        # the widest layout, 64 sequences, into 8 bits with a scale for each 128 columns for a product in 8 bits
        _norm("norm-8bit-large", 65536, 2048, out="e4m3"),
        # packed sequences of an odd width, fp32 throughout
        _norm("norm-odd", 4907, 771, x="f32", residual="f32", out="f32"),
        # a worker's batch of 8 full sequences (GPT-2 small), an fp32 residual stream
        _normback("normback-train", 8192, 768, h="f32", dx="f32"),
        # the widest layout from an 8-bit checkpoint; the normed rows again, for the next product's weight gradient
        _normback("normback-8bit-large", 65536, 2048, h="int8", again=True),
        # 25 images of 197 tokens, an odd width, rows apart: written in the forward pass, restored in the backward pass
        _checkpoint("checkpoint-odd", 25 * 197, 771, x="f32", code="e4m3", group=64, pad=5),
        # the hidden rows of GPT-2 medium, 16 sequences
        _checkpoint("checkpoint-large", 16384, 4096),
        # DeiT-Tiny's hidden rows of four images, fp32, nothing saved in 8 bits
        _act("act-small", 4 * 197, 768, x="f32", code="none"),
        # a gated block of the widest layout, forward and backward, x and up side by side as one product leaves them
        _act("act-gated-large", 16384, 8192, kind="silu", gated=True, fused=True),
        # one new token for each of 8 sequences at far positions of their own: latency
        _rotary("rotary-decode", 8, 1, 12, index="i64", first=100000, scaling="linear"),
        # a worker's batch, queries and keys where the fused product left them
        _rotary("rotary-train", 8, 1024, 12, fused=True),
        # long sequences scaled by parts, grouped keys, pairs side by side, the gradient
        _rotary("rotary-back-large", 4, 16384, 32, kv_heads=8, head_dim=128, rotary_dim=128, interleaved=True, scaling="parts",
                inverse=True),
    ]


def _log_int(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _width(rng, high):
    d = _log_int(rng, 64, high)
    return d if rng.random() < 0.3 else max(64, d // 64 * 64)


def draw(rng):
    top = {c["op"]: max(work(k)["bytes"] for k in listed() if k["op"] == c["op"]) for c in listed()}
    kind = lambda: "bf16" if rng.random() < 0.7 else "f32"  # noqa: E731
    while True:
        op = rng.choice(["norm", "normback", "checkpoint", "act", "rotary"])
        code, group = rng.choice(["int8", "e4m3"]), rng.choice([32, 64, 128, 128, 256])
        pad, rows = rng.choice([0, 0, 0, 64, 5]), _log_int(rng, 1, 65536)
        if op == "norm":
            c = _norm(None, rows, _width(rng, 8192), x=kind(), residual=rng.choice(["none", "f32", "bf16", "bf16"]),
                      out=rng.choice(["bf16", "bf16", "f32", "e4m3"]), weight=kind(), group=rng.choice([group, 0]), pad=pad)
        elif op == "normback":
            c = _normback(None, rows, _width(rng, 8192), dout=kind(), h=rng.choice(["bf16", "f32", code, code]),
                          group=rng.choice([group, 0]), residual=rng.random() < 0.7, dx=kind(), weight=kind(),
                          again=rng.random() < 0.4, pad=pad)
        elif op == "checkpoint":
            c = _checkpoint(None, rows, _width(rng, 8192), x=kind(), out=kind(), code=code, group=rng.choice([group, group, 0]), pad=pad)
        elif op == "act":
            c = _act(None, rows, _width(rng, 8192), x=kind(), kind=rng.choice(["silu", "gelu"]), gated=rng.random() < 0.6,
                     code=rng.choice(["none", code, code]), group=group, fused=rng.random() < 0.5)
        else:
            d = rng.choice([64, 64, 80, 128, 128, 256])
            c = _rotary(None, _log_int(rng, 1, 64), _log_int(rng, 1, 16384), _log_int(rng, 1, 32), head_dim=d,
                        kv_heads=_log_int(rng, 1, 16), rotary_dim=rng.choice([d, d, d // 2, d // 4]), x=kind(),
                        interleaved=rng.random() < 0.4, index=rng.choice(["none", "i32", "i64"]),
                        first=rng.choice([0, _log_int(rng, 1, 1 << 20)]), scaling=rng.choice(["none", "linear", "base", "parts"]),
                        inverse=rng.random() < 0.4, fused=rng.random() < 0.5)
        c.pop("name")
        if work(c)["bytes"] <= top[op]:
            return c


# ---- inputs ------------------------------------------------------------------

def _codes(x, code, group):
    """The codes of a matrix, as fp32 numbers, and the scales of its groups (0: one group a row).

    A group's largest magnitude a gives inv = top / a and scale = a * (1 / top); one below 2^-100 is held as zeros."""
    rows, cols = x.shape
    width = group or cols
    x = torch.nn.functional.pad(x.float(), (0, -cols % width)).view(rows, -1, width)
    a = x.abs().amax(-1, keepdim=True)
    inv = torch.where(a < 2.0 ** -100, torch.zeros_like(a), torch.full_like(a, TOPS[code]) / a)
    scale = torch.where(a < 2.0 ** -100, torch.zeros_like(a), a * float(np.float32(1 / TOPS[code])))
    q = x * inv
    q = q.round() if code == "int8" else q.to(torch.float8_e4m3fn).float()
    return q.view(rows, -1)[:, :cols], scale.view(rows, -1)


def _restored(codes, scales, group):
    cols = codes.shape[1]
    return codes.float() * scales.repeat_interleave(group or cols, 1)[:, :cols]


def _frequencies(case):
    """Radians a position for each pair, and the factor of all results."""
    R, base, factor, length = case["rotary_dim"], 10000.0, 8.0, 4096.0
    if case["scaling"] == "base":
        base = base * factor ** (R / (R - 2))
    f = [base ** (-2.0 * i / R) for i in range(R // 2)]
    if case["scaling"] == "linear":
        f = [v / factor for v in f]
    if case["scaling"] == "parts":  # turns within the old length: all of the frequency from 32 on, 1 / factor of it up to 1
        share = [min(1.0, max(0.0, (length * v / (2 * math.pi) - 1.0) / 31.0)) for v in f]
        f = [v * (s + (1 - s) / factor) for v, s in zip(f, share)]
        return f, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 29)

    def normal(shape, kind, std=1.0, pad=0):
        x = torch.randn(*shape[:-1], shape[-1] + pad, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(TYPES[kind])
        return x[..., :shape[-1]]

    def activations(shape, kind, pad=0):  # some columns are much larger than the rest, as activations have them
        x = torch.randn(*shape[:-1], shape[-1] + pad, generator=g, device="cuda")[..., :shape[-1]]
        big = torch.rand(shape[-1], generator=g, device="cuda") < 0.01
        x.mul_(torch.where(big, 12.0, 1.0))
        return x if kind == "f32" else x.to(TYPES[kind])

    empty = lambda shape, kind: torch.empty(*shape, dtype=TYPES[kind], device="cuda")  # noqa: E731
    s, op = {"case": case}, case["op"]
    if op == "rotary":
        B, S, H, K, D = (case[k] for k in ("batch", "seq", "heads", "kv_heads", "head_dim"))
        if case["fused"]:  # queries, keys and values side by side
            whole = normal((B, S, H + 2 * K, D), case["x"])
            s["q"], s["k"] = whole[:, :, :H], whole[:, :, H:H + K]
        else:
            s["q"], s["k"] = normal((B, S, H, D), case["x"]), normal((B, S, K, D), case["x"])
        s["q_out"], s["k_out"] = empty((B, S, H, D), case["x"]), empty((B, S, K, D), case["x"])
        s["positions"] = None
        if case["index"] != "none":  # each sequence begins at a place of its own
            begin = torch.randint(case["first"], 2 * case["first"] + 2, (B, 1), generator=g, device="cuda")
            s["positions"] = (begin + torch.arange(S, device="cuda")).to(torch.int32 if case["index"] == "i32" else torch.int64)
        frequencies, s["magnitude"] = _frequencies(case)
        s["frequencies"] = torch.tensor(frequencies, dtype=torch.float64, device="cuda")
        if own:
            from communication_compressed_sign_gb300 import Rotary, RotaryScaling
            scaling = {"none": None, "linear": RotaryScaling("linear", 8.0), "base": RotaryScaling("base", 8.0),
                       "parts": RotaryScaling("parts", 8.0, length=4096)}[case["scaling"]]
            s["rotary"] = Rotary(D, rotary_dim=case["rotary_dim"], base=10000.0, interleaved=case["interleaved"], scaling=scaling)
        return s
    n, D = case["rows"], case["dim"]
    if op == "act":
        if case["fused"] and case["gated"]:
            whole = activations((n, 2 * D), case["x"])
            s["x"], s["up"] = whole[:, :D], whole[:, D:]
            both = empty((n, 2 * D), case["x"])
            s["dx"], s["dup"] = both[:, :D], both[:, D:]
        else:
            s["x"], s["dx"] = activations((n, D), case["x"]), empty((n, D), case["x"])
            s["up"], s["dup"] = (activations((n, D), case["x"]), empty((n, D), case["x"])) if case["gated"] else (None, None)
        s["dout"] = normal((n, D), case["x"], 1e-2)
        s["out"] = empty((n, D), case["x"])
        if case["code"] != "none":
            s["again"] = empty((n, D), case["x"])
            if own:
                from communication_compressed_sign_gb300 import Packed
                s["saved"] = Packed.empty((n, D), group=case["group"], dtype=TYPES[case["code"]])
                s["saved_up"] = Packed.empty((n, D), group=case["group"], dtype=TYPES[case["code"]]) if case["gated"] else None
        return s
    if op == "checkpoint":
        s["x"] = activations((n, D), case["x"], case["pad"])
        s["out"] = empty((n, D), case["out"])
        if own:
            from communication_compressed_sign_gb300 import Packed
            s["saved"] = Packed.empty((n, D), group=case["group"], dtype=TYPES[case["code"]])
        return s
    s["weight"] = (1.0 + normal((D,), "f32", 0.1)).to(TYPES[case["weight"]])
    if own:
        from communication_compressed_sign_gb300 import Packed, RmsNorm
        s["norm"] = RmsNorm(D, eps=EPS)
    if op == "norm":
        s["x"] = activations((n, D), case["x"], case["pad"])
        s["residual"] = activations((n, D), case["residual"], case["pad"]) if case["residual"] != "none" else None
        s["summed"] = empty((n, D), case["residual"]) if case["residual"] != "none" else None
        s["rstd"] = torch.empty(n, device="cuda")
        if case["out"] != "e4m3":
            s["out"] = empty((n, D), case["out"])
        elif own:
            s["out"] = Packed.empty((n, D), group=case["group"], dtype=TYPES["e4m3"])
        return s
    h = activations((n, D), "f32" if case["h"] in TOPS else case["h"], case["pad"])
    s["rstd"] = (h.float().square().mean(-1) + EPS).rsqrt()
    if case["h"] in TOPS:
        codes, scales = _codes(h, case["h"], case["group"])
        s["h"] = (codes.to(TYPES[case["h"]]).contiguous(), scales.contiguous())
        if own:
            s["packed"] = Packed(*s["h"], group=case["group"])
    else:
        s["h"] = h
    s["dout"] = normal((n, D), case["dout"], 1e-3, case["pad"])
    s["residual_grad"] = normal((n, D), case["dx"], 1e-3, case["pad"]) if case["residual"] else None
    s["dx"], s["dw"] = empty((n, D), case["dx"]), empty((D,), case["weight"])
    s["again"] = empty((n, D), case["dout"]) if case["again"] else None
    return s


# ---- one pass ------------------------------------------------------------------

def _plain_norm(s, case):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    r = (h.square().mean(-1) + EPS).rsqrt()
    y = h * r[:, None] * s["weight"].float()
    got = {"rstd": r}
    if s["residual"] is not None:
        got["summed"] = h.to(TYPES[case["residual"]])
    if case["out"] == "e4m3":
        codes, got["scales"] = _codes(y, "e4m3", case["group"])
        return {**got, "codes": codes.to(torch.float8_e4m3fn)}
    return {**got, "out": y.to(TYPES[case["out"]])}


def _own_norm(s, case):
    s["norm"].forward(s["x"], s["weight"], residual=s["residual"], summed=s["summed"], rstd=s["rstd"], out=s["out"])
    got = {"rstd": s["rstd"]}
    if s["residual"] is not None:
        got["summed"] = s["summed"]
    if case["out"] == "e4m3":
        return {**got, "scales": s["out"].scales, "codes": s["out"].codes}
    return {**got, "out": s["out"]}


def _plain_normback(s, case):
    h = _restored(*s["h"], case["group"]) if case["h"] in TOPS else s["h"].float()
    r = s["rstd"][:, None]
    dout, n = s["dout"].float(), h * r
    g = dout * s["weight"].float()
    dx = r * (g - n * (g * n).mean(-1, keepdim=True))
    if s["residual_grad"] is not None:
        dx = dx + s["residual_grad"].float()
    got = {"dx": dx.to(TYPES[case["dx"]]), "dw": (dout * n).sum(0).to(TYPES[case["weight"]])}
    if case["again"]:
        got["again"] = (n * s["weight"].float()).to(TYPES[case["dout"]])
    return got


def _own_normback(s, case):
    s["norm"].backward(s["dout"], s["packed"] if case["h"] in TOPS else s["h"], s["rstd"], s["weight"],
                       residual_grad=s["residual_grad"], out=s["dx"], weight_grad=s["dw"], again=s["again"])
    return {"dx": s["dx"], "dw": s["dw"]} if s["again"] is None else {"dx": s["dx"], "dw": s["dw"], "again": s["again"]}


def _plain_checkpoint(s, case):
    return _restored(*_codes(s["x"], case["code"], case["group"]), case["group"]).to(TYPES[case["out"]])


def _own_checkpoint(s, case):
    from communication_compressed_sign_gb300 import pack8, unpack8
    return unpack8(pack8(s["x"], out=s["saved"]), out=s["out"])


def _value_and_slope(x, kind):
    """The activation and its derivative: x * sigmoid(z), z = x or 2 sqrt(2 / pi) (x + 0.044715 x^3)."""
    if kind == "silu":
        z, dz = x, 1.0
    else:
        k = 2.0 * math.sqrt(2.0 / math.pi)
        z, dz = k * (x + 0.044715 * x * x * x), k * (1.0 + 3 * 0.044715 * x * x)
    t = 1.0 / (1.0 + torch.exp(-z))
    return x * t, t + x * t * (1.0 - t) * dz


def _plain_act(s, case):
    x, up, dout, to = s["x"].float(), s["up"], s["dout"].float(), TYPES[case["x"]]
    out = _value_and_slope(x, case["kind"])[0]
    if up is not None:
        up = up.float()
        out = out * up
    if case["code"] != "none":
        x = _restored(*_codes(x, case["code"], case["group"]), case["group"])
        if up is not None:
            up = _restored(*_codes(up, case["code"], case["group"]), case["group"])
    f, slope = _value_and_slope(x, case["kind"])
    got = {"out": out.to(to), "dx": (dout * slope if up is None else dout * up * slope).to(to)}
    if up is not None:
        got["dup"] = (dout * f).to(to)
    if case["code"] != "none":
        got["again"] = (f if up is None else f * up).to(to)
    return got


def _own_act(s, case):
    from communication_compressed_sign_gb300 import activation, activation_backward
    got = {"out": s["out"], "dx": s["dx"]}
    if case["gated"]:
        got["dup"] = s["dup"]
    if case["code"] == "none":
        activation(s["x"], s["up"], kind=case["kind"], out=s["out"])
        activation_backward(s["dout"], s["x"], s["up"], kind=case["kind"], dx=s["dx"], dup=s["dup"])
        return got
    activation(s["x"], s["up"], kind=case["kind"], out=s["out"], saved=s["saved"], saved_up=s["saved_up"])
    activation_backward(s["dout"], s["saved"], s["saved_up"], kind=case["kind"], dx=s["dx"], dup=s["dup"], again=s["again"])
    return {**got, "again": s["again"]}


def _plain_rotated(x, cos, sin, case):
    R, to = case["rotary_dim"], x.dtype
    x = x.float()
    turned, rest = x[..., :R], x[..., R:]
    if case["interleaved"]:
        a, b = turned[..., 0::2], turned[..., 1::2]
        both = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = turned[..., :R // 2], turned[..., R // 2:]
        both = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([both, rest], -1).to(to)


def _plain_rotary(s, case):
    p = s["positions"]
    if p is None:
        p = (torch.arange(case["seq"], device="cuda") + case["first"])[None, :]
    angle = p.double()[..., None, None] * s["frequencies"]
    m = s["magnitude"]
    cos, sin = (torch.cos(angle) * m).float(), (torch.sin(angle) * (-m if case["inverse"] else m)).float()
    return {"q": _plain_rotated(s["q"], cos, sin, case), "k": _plain_rotated(s["k"], cos, sin, case)}


def _own_rotary(s, case):
    go = s["rotary"].backward if case["inverse"] else s["rotary"].forward
    go(s["q"], s["k"], positions=s["positions"], first_position=case["first"], q_out=s["q_out"], k_out=s["k_out"])
    return {"q": s["q_out"], "k": s["k_out"]}


def run(state):
    case = state["case"]
    if own:
        return {"norm": _own_norm, "normback": _own_normback, "checkpoint": _own_checkpoint, "act": _own_act,
                "rotary": _own_rotary}[case["op"]](state, case)
    return {"norm": _plain_norm, "normback": _plain_normback, "checkpoint": _plain_checkpoint, "act": _plain_act,
            "rotary": _plain_rotary}[case["op"]](state, case)


# ---- what a pass cannot do without ----------------------------------------------

def _packed_bytes(case, n, D):
    return n * D + n * 4 * (-(-D // (case["group"] or D)))


def work(case):
    if case["op"] == "rotary":
        places = case["batch"] * case["seq"]
        heads = places * (case["heads"] + case["kv_heads"])
        return {"bytes": 2 * heads * case["head_dim"] * SIZES[case["x"]] + places * SIZES[case["index"]],
                "flops": heads * case["rotary_dim"] * 3}
    n, D = case["rows"], case["dim"]
    if case["op"] == "norm":
        out = _packed_bytes(case, n, D) if case["out"] == "e4m3" else n * D * SIZES[case["out"]]
        return {"bytes": n * D * (SIZES[case["x"]] + 2 * SIZES[case["residual"]]) + out + 4 * n + D * SIZES[case["weight"]],
                "flops": n * D * 5}
    if case["op"] == "normback":
        h = _packed_bytes(case, n, D) if case["h"] in TOPS else n * D * SIZES[case["h"]]
        each = SIZES[case["dout"]] * (2 if case["again"] else 1) + SIZES[case["dx"]] * (2 if case["residual"] else 1)
        return {"bytes": n * D * each + h + 4 * n + 2 * D * SIZES[case["weight"]], "flops": n * D * 10}
    if case["op"] == "checkpoint":
        return {"bytes": n * D * (SIZES[case["x"]] + SIZES[case["out"]]) + 2 * _packed_bytes(case, n, D), "flops": n * D * 3}
    inputs, one = 2 if case["gated"] else 1, n * D * SIZES[case["x"]]
    if case["code"] == "none":  # forward: inputs and out; backward: inputs, dout and gradients
        return {"bytes": one * (3 * inputs + 2), "flops": n * D * (15 + 5 * inputs)}
    return {"bytes": one * (2 * inputs + 3) + 2 * inputs * _packed_bytes(case, n, D), "flops": n * D * (20 + 10 * inputs)}


# ---- the definition in 64 bits ---------------------------------------------------

def _exact_values(x, code, group):
    """What the codes of x stand for."""
    n, cols = x.shape
    width = group or cols
    out = torch.empty_like(x)
    for first in range(0, cols, max(width, 1)):
        part = x[:, first:first + width]
        unit = part.abs().amax(1, keepdim=True) / TOPS[code]
        q = torch.where(unit > 0, part / unit, torch.zeros_like(part))
        if code == "int8":
            q = torch.round(q)
        else:  # three bits behind the leading one, 2^-9 the smallest step
            step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
            q = torch.round(q / step) * step
        out[:, first:first + width] = q * unit
    return out


def _exact_act(x, kind):
    """f and f' by the hyperbolic tangent."""
    if kind == "silu":
        t = 0.5 * (1 + torch.tanh(x / 2))
        return x * t, t * (1 + x * (1 - t))
    w = math.sqrt(2 / math.pi)
    t = torch.tanh(w * (x + 0.044715 * x ** 3))
    return 0.5 * x * (1 + t), 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * w * (1 + 0.134145 * x * x)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "rotary":
        B, S, R = case["batch"], case["seq"], case["rotary_dim"]
        f, m = _frequencies(case)
        p = s["positions"]
        p = torch.arange(case["first"], case["first"] + S, device="cuda").expand(B, S) if p is None else p
        turn = torch.polar(torch.full((), m, dtype=torch.float64, device="cuda"),
                           p.to(torch.float64).reshape(B, S, 1, 1) * torch.tensor(f, dtype=torch.float64, device="cuda"))
        turn = turn.conj() if case["inverse"] else turn
        got = {}
        for name in ("q", "k"):
            x = s[name].double()
            y = x.clone()
            first, second = (slice(0, R, 2), slice(1, R, 2)) if case["interleaved"] else (slice(0, R // 2), slice(R // 2, R))
            z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
            y[..., first], y[..., second] = z.real, z.imag
            got[name] = y
        return got
    if op == "checkpoint":
        return _exact_values(s["x"].double(), case["code"], case["group"])
    if op == "act":
        x, up, dout = s["x"].double(), None if s["up"] is None else s["up"].double(), s["dout"].double()
        f, _ = _exact_act(x, case["kind"])
        got = {"out": f if up is None else f * up}
        if case["code"] != "none":
            x = _exact_values(x, case["code"], case["group"])
            up = None if up is None else _exact_values(up, case["code"], case["group"])
        f, slope = _exact_act(x, case["kind"])
        got["dx"] = dout * slope * (1.0 if up is None else up)
        if up is not None:
            got["dup"] = dout * f
        if case["code"] != "none":
            got["again"] = f if up is None else f * up
        return got
    w, D = s["weight"].double(), case["dim"]
    if op == "norm":
        h = s["x"].double()
        got = {}
        if s["residual"] is not None:
            h = h + s["residual"].double()
            got["summed"] = h
        norm = torch.sqrt(torch.einsum("ij,ij->i", h, h) / D + EPS)
        got["rstd"] = 1 / norm
        y = h / norm[:, None] * w
        if case["out"] != "e4m3":
            return {**got, "out": y}
        width = case["group"] or D
        scales = torch.stack([part.abs().amax(1) for part in y.split(width, 1)], 1) / TOPS["e4m3"]
        return {**got, "scales": scales, "codes": torch.cat([part / scales[:, i:i + 1] for i, part in enumerate(y.split(width, 1))], 1)}
    if case["h"] in TOPS:
        codes, scales = s["h"]
        width = case["group"] or D
        h = torch.cat([part.float().double() * scales[:, i:i + 1].double() for i, part in enumerate(codes.split(width, 1))], 1)
    else:
        h = s["h"].double()
    r, dout = s["rstd"].double(), s["dout"].double()
    along = torch.einsum("ij,j,ij->i", dout, w, h) * r ** 3 / D
    dx = dout * w * r[:, None] - h * along[:, None]
    if s["residual_grad"] is not None:
        dx = dx + s["residual_grad"].double()
    got = {"dx": dx, "dw": torch.einsum("ij,ij,i->j", dout, h, r)}
    if case["again"]:
        got["again"] = h * r[:, None] * w
    return got
