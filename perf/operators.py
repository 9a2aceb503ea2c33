"""The 8-bit operators of the codec, as cases to be measured.

Three operators that a W8A8 linear layer consists of:

  quant8    rows -> int8 codes with one fp32 scale a row (weights with their channel scale, activations,
            gated activations), and read back with dequant8;
  rmsnorm8  residual addition and root-mean-square norm, with the normalized rows as int8 codes and scales;
  gemm8     the product of int8 activations (a scale for each token) and int8 weights (a scale for each
            output channel).

Codes have a row pitch that is a multiple of 16 bytes.  Where an operator gives codes, the case reads them
back, and returns the values that they stand for, as bf16.

listed() and draw() give cases, prepare() their inputs, run() one pass: in elementary torch operations, or,
with `own` set, through the package.
"""
import math

import torch

own = False

# Widths and layer shapes (outputs x inputs) that the benchmark and the tests of this repository use.
WIDTHS = (4096, 5120, 11008, 13824)
EPS = 1e-5


def listed():
    return [
        # the input of one token's attention output projection
        dict(name="quant8 1x5120", op="quant8", rows=1, cols=5120, dtype="bf16", gate=False, scale=False),
        # a weight matrix of an MLP, with its activation-aware channel scale
        dict(name="quant8 weights 13824x5120", op="quant8", rows=13824, cols=5120, dtype="bf16", gate=False, scale=True),
        # gate and up halves of one product's output, for a prompt of 2048 tokens, before the down projection
        dict(name="quant8 gated 2048x13824", op="quant8", rows=2048, cols=13824, dtype="bf16", gate=True, scale=False),
        # a small fp32 matrix with a width that no vector load divides
        dict(name="quant8 fp32 333x1003", op="quant8", rows=333, cols=1003, dtype="fp32", gate=False, scale=True),
        # one token between two sublayers
        dict(name="rmsnorm8 1x4096", op="rmsnorm8", rows=1, cols=4096, dtype="bf16", residual=True),
        # a prompt of 4096 tokens between two sublayers
        dict(name="rmsnorm8 4096x5120", op="rmsnorm8", rows=4096, cols=5120, dtype="bf16", residual=True),
        # the first norm of a stack (nothing to add), fp32, a ragged batch
        dict(name="rmsnorm8 fp32 515x4100", op="rmsnorm8", rows=515, cols=4100, dtype="fp32", residual=False),
        # one token through a square projection: a read of the weights
        dict(name="gemm8 1x5120x5120", op="gemm8", rows=1, cols=5120, inner=5120, out="bf16"),
        # a decoding batch of 16 through an MLP's up projection
        dict(name="gemm8 16x13824x5120", op="gemm8", rows=16, cols=13824, inner=5120, out="bf16"),
        # a ragged batch through a down projection
        dict(name="gemm8 77x4096x11008", op="gemm8", rows=77, cols=4096, inner=11008, out="fp32"),
        # a prompt through a square projection
        dict(name="gemm8 1500x5120x5120", op="gemm8", rows=1500, cols=5120, inner=5120, out="bf16"),
        # a batch of prompts through an MLP's up projection
        dict(name="gemm8 8192x13824x5120", op="gemm8", rows=8192, cols=13824, inner=5120, out="bf16"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _width(rng, low, high):
    """A width: one of the models', a multiple of 64, or any number."""
    kind = rng.random()
    if kind < 0.3:
        return rng.choice([w for w in WIDTHS if low <= w <= high])
    w = _log(rng, low, high)
    return max(64, w // 64 * 64) if kind < 0.7 else w


def draw(rng):
    op = rng.choice(("quant8", "rmsnorm8", "gemm8", "gemm8"))
    if op == "quant8":
        return dict(op=op, rows=_log(rng, 1, 8192), cols=_width(rng, 64, 13824), dtype=rng.choice(("bf16", "fp32")),
                    gate=rng.random() < 0.4, scale=rng.random() < 0.4)
    if op == "rmsnorm8":
        return dict(op=op, rows=_log(rng, 1, 8192), cols=_width(rng, 64, 8192), dtype=rng.choice(("bf16", "bf16", "fp32")),
                    residual=rng.random() < 0.7)
    while True:
        m, n, k = _log(rng, 1, 8192), _width(rng, 64, 13824), _width(rng, 64, 13824)
        if m * n * k <= 8192 * 13824 * 5120:
            return dict(op=op, rows=m, cols=n, inner=k, out=rng.choice(("bf16", "bf16", "fp32")))


def _dtype(name):
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[name]


def _codes(rows, cols, gen):
    """Codes and scales of rows * cols Gaussian values, as a quantizer leaves them: each row's largest value
    at 127, row pitch a multiple of 16 bytes."""
    x = torch.randn((rows, cols), generator=gen, device="cuda")
    top = x.abs().amax(1, keepdim=True)
    pitch = (cols + 15) // 16 * 16
    q = torch.zeros((rows, pitch), dtype=torch.int8, device="cuda")[:, :cols]
    q.copy_(torch.round(x * (127.0 / top)))
    return q, (top[:, 0] / 127.0)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rows, cols = case["rows"], case["cols"]
    if case["op"] == "gemm8":
        xq, xs = _codes(rows, case["inner"], gen)
        wq, ws = _codes(cols, case["inner"], gen)
        # tokens differ in size; weights are small
        xs = xs * torch.exp(torch.randn((rows,), generator=gen, device="cuda"))
        return dict(case, xq=xq, xs=xs, wq=wq, ws=ws * 0.02)
    dt = _dtype(case["dtype"])
    # a few channels of activations are many times larger than the others
    chan = torch.exp(0.5 * torch.randn((cols,), generator=gen, device="cuda"))
    chan[torch.randint(0, cols, (max(1, cols // 512),), generator=gen, device="cuda")] *= 10.0
    state = dict(case)
    if case["op"] == "quant8":
        if case["gate"]:
            both = torch.randn((rows, 2 * cols), generator=gen, device="cuda")
            both[:, cols:] *= chan
            both = both.to(dt)
            state.update(gate=both[:, :cols], x=both[:, cols:])
        else:
            state.update(gate=None, x=(torch.randn((rows, cols), generator=gen, device="cuda") * chan).to(dt))
        state["scale"] = chan.pow(-0.3) if case["scale"] else None
        return state
    x = torch.randn((rows, cols), generator=gen, device="cuda")
    state["residual"] = (4 * torch.randn((rows, cols), generator=gen, device="cuda") * chan).to(dt) if case["residual"] else None
    state["x"] = x.to(dt)
    state["weight"] = 1.0 + 0.1 * torch.randn((cols,), generator=gen, device="cuda")
    return state


def _quantize(a):
    """Values of the rows of fp32 `a` in 8 bits, and the rows' scales."""
    top = a.abs().amax(1, keepdim=True)
    step = top / 127.0
    back = torch.where(top > 0, 127.0 / top, torch.zeros_like(top))
    return torch.round(a * back) * step, step[:, 0]


def _plain(s):
    if s["op"] == "gemm8":
        y = torch.mm(s["xq"].float(), s["wq"].float().t())
        return {"y": (y * s["xs"][:, None] * s["ws"]).to(_dtype(s["out"]))}
    if s["op"] == "quant8":
        a = s["x"].float()
        if s["gate"] is not None:
            g = s["gate"].float()
            a = a * (g / (1.0 + torch.exp(-g)))
        if s["scale"] is not None:
            a = a * s["scale"]
        v, step = _quantize(a)
        if s["scale"] is not None:
            v = v / s["scale"]
        return {"row_scale": step, "values": v.to(torch.bfloat16)}
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["weight"]
    v, step = _quantize(y)
    out = {"row_scale": step, "values": v.to(torch.bfloat16)}
    if s["residual"] is not None:
        out["sum"] = h.to(s["x"].dtype)
    return out


def _own(s):
    import weight_quantization_codec_amd as q
    if s["op"] == "gemm8":
        return {"y": q.gemm8(s["xq"], s["xs"], s["wq"], s["ws"], out_dtype=_dtype(s["out"]))}
    if s["op"] == "quant8":
        codes, row_scale = q.quant8(s["x"], scale=s["scale"], gate=s["gate"])
        return {"row_scale": row_scale, "values": q.dequant8(codes, row_scale, scale=s["scale"])}
    codes, row_scale, h = q.rmsnorm8(s["x"], s["weight"], eps=EPS, residual=s["residual"])
    out = {"row_scale": row_scale, "values": q.dequant8(codes, row_scale)}
    if s["residual"] is not None:
        out["sum"] = h
    return out


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    n, m = case["rows"], case["cols"]
    if case["op"] == "gemm8":
        k = case["inner"]
        return {"bytes": n * k + m * k + 4 * (n + m) + n * m * (2 if case["out"] == "bf16" else 4), "flops": 2 * n * m * k}
    size = 2 if case["dtype"] == "bf16" else 4
    # the rows, their codes and scales, and the values read back
    moved = n * m * (size + 1 + 2) + 4 * n
    if case["op"] == "quant8":
        moved += (n * m * size if case["gate"] else 0) + (4 * m if case["scale"] else 0)
    else:
        moved += (2 * n * m * size if case["residual"] else 0) + 4 * m
    return {"bytes": moved, "flops": 8 * n * m}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "gemm8":
        # sums of up to 1024 products of codes are whole numbers below 2^24: each such piece is exact in
        # fp32, in any order, and the pieces are added in fp64
        k, xq, wq = case["inner"], s["xq"], s["wq"]
        total = torch.zeros((case["rows"], case["cols"]), dtype=torch.float64, device="cuda")
        for at in range(0, k, 1024):
            total += torch.mm(xq[:, at:at + 1024].float(), wq[:, at:at + 1024].float().t()).double()
        return {"y": total.mul_(s["xs"].double()[:, None]).mul_(s["ws"].double())}
    values, scales, sums = [], [], []
    gate, residual = s.get("gate"), s.get("residual")
    for at in range(0, case["rows"], 1024):   # a block of rows at a time: fp64 is large
        a = s["x"][at:at + 1024].double()
        if case["op"] == "quant8":
            if gate is not None:
                g = gate[at:at + 1024].double()
                a = a * g * torch.sigmoid(g)
            chan = s["scale"].double() if s["scale"] is not None else torch.ones((), dtype=torch.float64, device="cuda")
            a = a * chan
        else:
            if residual is not None:
                a = a + residual[at:at + 1024].double()
                sums.append(a)
            chan = torch.ones((), dtype=torch.float64, device="cuda")
            a = a / torch.sqrt(torch.sum(a ** 2, 1, keepdim=True) / case["cols"] + EPS) * s["weight"].double()
        step = torch.max(torch.abs(a), 1, keepdim=True).values / 127
        scales.append(step[:, 0])
        values.append(torch.where(step > 0, torch.round(a / step), 0.0) * step / chan)
    out = {"row_scale": torch.cat(scales), "values": torch.cat(values)}
    if sums:
        out["sum"] = torch.cat(sums)
    return out
