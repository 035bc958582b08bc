"""Measured cases of the operators of a quantized linear layer.

Four kinds of pass over dual-scale microscaled operands (W ~ D_a Q D_b, the column inverse scales b folded
into the activations before they are quantized):

* ``matmul``  Y = s_x s_w (a_x q_x)(a_w q_w)^T of quantized activations and a quantized weight matrix;
* ``norm``    residual addition, root-mean-square norm, times b, quantized to MXFP8;
* ``glu``     silu(gate) * up, times b, quantized to MXFP8;
* ``mlp``     the four calls of an MLP block in a row: norm, gate/up product, glu, down product.

With ``own`` false a pass is elementary torch operations; with ``own`` true it is the calls that a user makes
of the package.  Formats: NVFP4 (E2M1 codes, E4M3 scales per 16, one fp32 tensor scale), MXFP4 (E2M1 codes,
power-of-two scales per 32) and MXFP8 (E4M3 codes, power-of-two scales per 32).
"""
import math

import torch

own = False

EPS = 1e-5
GROUP = {"nvfp4": 16, "mxfp4": 32, "mxfp8": 32}
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
LARGEST = 8192 * 14336 * 4096  # multiply-adds of the largest listed product


# ---------------------------------------------------------------------------
# Cases

def listed():
    return [
        # one request decoding: the attention output projection of one token, where latency counts
        {"name": "matmul_nvfp4_1tok_4096x4096", "op": "matmul", "fmt": "nvfp4", "tokens": 1, "rows": 4096, "cols": 4096,
         "dtype": "bf16"},
        # a small decode batch through the down projection (long sums, few outputs)
        {"name": "matmul_mxfp4_16tok_4096x14336", "op": "matmul", "fmt": "mxfp4", "tokens": 16, "rows": 4096,
         "cols": 14336, "dtype": "f16"},
        # a ragged prompt through a key projection, summed on in fp32 by its caller
        {"name": "matmul_mxfp8_333tok_1024x4096", "op": "matmul", "fmt": "mxfp8", "tokens": 333, "rows": 1024,
         "cols": 4096, "dtype": "f32"},
        # no size a multiple of a tile, scale rows at odd byte offsets
        {"name": "matmul_nvfp4_1000tok_1001x1056", "op": "matmul", "fmt": "nvfp4", "tokens": 1000, "rows": 1001,
         "cols": 1056, "dtype": "bf16"},
        # a prompt batch through the down projection with 8-bit operands
        {"name": "matmul_mxfp8_4096tok_4096x14336", "op": "matmul", "fmt": "mxfp8", "tokens": 4096, "rows": 4096,
         "cols": 14336, "dtype": "bf16"},
        # the largest: a prefill batch through the gate (or up) projection
        {"name": "matmul_nvfp4_8192tok_14336x4096", "op": "matmul", "fmt": "nvfp4", "tokens": 8192, "rows": 14336,
         "cols": 4096, "dtype": "bf16"},
        # the norm before a projection, one token and a prefill batch
        {"name": "norm_mxfp8_1tok_4096", "op": "norm", "fmt": "mxfp8", "tokens": 1, "cols": 4096, "dtype": "bf16",
         "residual": True},
        {"name": "norm_mxfp8_8192tok_4096", "op": "norm", "fmt": "mxfp8", "tokens": 8192, "cols": 4096,
         "dtype": "bf16", "residual": True},
        # the activation of an MLP between its two products, a decode batch and a prefill batch
        {"name": "glu_mxfp8_16tok_14336", "op": "glu", "fmt": "mxfp8", "tokens": 16, "cols": 14336, "dtype": "bf16"},
        {"name": "glu_mxfp8_8192tok_14336", "op": "glu", "fmt": "mxfp8", "tokens": 8192, "cols": 14336,
         "dtype": "bf16"},
        # a whole MLP block: one decoded token, and a prompt
        {"name": "mlp_nvfp4_1tok_4096_14336", "op": "mlp", "fmt": "nvfp4", "tokens": 1, "cols": 4096, "inter": 14336,
         "dtype": "bf16"},
        {"name": "mlp_mxfp4_1500tok_4096_14336", "op": "mlp", "fmt": "mxfp4", "tokens": 1500, "cols": 4096,
         "inter": 14336, "dtype": "bf16"},
    ]


def draw(rng):
    def log(lo, hi, step=1):
        return max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi))) // step * step))

    op = rng.choice(["matmul", "matmul", "norm", "glu", "mlp"])
    case = {"op": op, "fmt": rng.choice(["nvfp4", "mxfp4", "mxfp8"]) if op in ("matmul", "mlp") else "mxfp8"}
    if op == "matmul":
        case.update(tokens=log(1, 8192), rows=log(64, 14336), cols=log(64, 14336, 32),
                    dtype=rng.choice(["bf16", "f16", "f32"]))
        case["tokens"] = max(1, min(case["tokens"], LARGEST // (case["rows"] * case["cols"])))
    elif op == "mlp":
        case.update(tokens=log(1, 1500), cols=log(64, 4096, 32), inter=log(64, 14336, 32), dtype="bf16")
    elif op == "norm":
        case.update(tokens=log(1, 8192), cols=log(64, 4096, 32), dtype=rng.choice(["bf16", "f16"]),
                    residual=rng.random() < 0.75)
    else:
        case.update(tokens=log(1, 8192), cols=log(64, 14336, 32), dtype=rng.choice(["bf16", "f16"]))
    return case


def work(case):
    """Every operand read once and every output written once; products are 2 T N K operations."""
    t, k = case["tokens"], case["cols"]
    es = 4 if case["dtype"] == "f32" else 2

    def quantized(r, c):
        return r * c // (1 if case["fmt"] == "mxfp8" else 2) + r * (c // GROUP[case["fmt"]])

    if case["op"] == "matmul":
        n = case["rows"]
        return {"bytes": quantized(t, k) + quantized(n, k) + t * n * es, "flops": 2 * t * n * k}
    if case["op"] == "norm":
        return {"bytes": t * k * es * (3 if case["residual"] else 1) + quantized(t, k) + 4 * k, "flops": 6 * t * k}
    if case["op"] == "glu":
        return {"bytes": t * k * es * 2 + quantized(t, k) + 2 * k, "flops": 8 * t * k}
    n = case["inter"]
    # the hidden state, its residual and the sum, the two weight matrices, the two outputs; what passes between the
    # four calls need not leave the chip
    return {"bytes": 3 * t * k * es + quantized(2 * n, k) + quantized(k, n) + t * k * es, "flops": 6 * t * n * k}


# ---------------------------------------------------------------------------
# Plain quantization (64 bits: decisions next to a border) and its inverse

def _nearest_pow2(v):
    """Nearest power of two in linear distance, 1.5 * 2^k up, within 2^-126 .. 2^126."""
    m, e = torch.frexp(v)  # v = m 2^e, m in [0.5, 1)
    e = (e - 1 + (m >= 0.75).to(e.dtype)).clamp(-126, 126)
    return torch.ldexp(torch.ones_like(v), e)


def _round_e4m3(m):
    """Magnitudes to the nearest E4M3 value, ties to the even mantissa, 448 at most."""
    _, e = torch.frexp(m)
    step = torch.ldexp(torch.ones_like(m), (e - 1).clamp(min=-6) - 3)
    return (torch.round(m / step) * step).clamp(max=448.0)


def _round_e2m1(m):
    """Magnitudes to the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6, ties to the even mantissa."""
    _, e = torch.frexp(m)
    step = torch.ldexp(torch.ones_like(m), (e - 1).clamp(0, 2) - 1)
    return (torch.round(m / step) * step).clamp(max=6.0)


def _bytes_of_e4m3(v):
    return v.to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8)


def _quantize(x, fmt):
    """x (fp64 [rows, cols]) in the format: absmax scales projected onto the format's set, nearest codes."""
    rows, cols = x.shape
    g = x.view(rows, cols // GROUP[fmt], GROUP[fmt])
    top = g.abs().amax(2)
    one = torch.ones((), dtype=x.dtype, device=x.device)
    if fmt == "nvfp4":
        tensor_scale = (top.amax() / 2688.0).to(torch.float32)
        tensor_scale = torch.where(top.amax() == 0, torch.ones_like(tensor_scale), tensor_scale)
        e = _round_e4m3(top / 6.0 / tensor_scale.double()).clamp(min=2.0 ** -9)
        e = torch.where(top == 0, one, e)
        scale, stored = e * tensor_scale.double(), _bytes_of_e4m3(e)
    else:
        tensor_scale = torch.ones((), device=x.device)
        scale = torch.where(top == 0, one, _nearest_pow2(top / (448.0 if fmt == "mxfp8" else 6.0)))
        stored = (torch.frexp(scale)[1] + 126).to(torch.uint8)
    m = g.abs() / scale.unsqueeze(2)
    if fmt == "mxfp8":
        q = _round_e4m3(m)
        codes = torch.where(q == 0, q, torch.copysign(q, g)).to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        q = _round_e2m1(m)
        c = (2 * q - (q - 2).clamp(min=0) - 0.5 * (q - 4).clamp(min=0)).to(torch.uint8)  # 0 .. 7
        c = c + 8 * ((g < 0) & (q > 0)).to(torch.uint8)
        codes = c.view(rows, cols // 2, 2)
        codes = codes[:, :, 0] + 16 * codes[:, :, 1]
    return {"codes": codes.reshape(rows, -1), "block_scales": stored, "tensor_scale": tensor_scale.reshape(1)}


def _values(t, fmt):
    """a q of a quantized matrix in fp32 (exact), without the tensor scale."""
    rows = t["codes"].shape[0]
    if fmt == "mxfp8":
        q = t["codes"].view(torch.float8_e4m3fn).to(torch.float32)
    else:
        table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=t["codes"].device)
        table = torch.cat([table, -table])
        c = t["codes"].to(torch.int32)
        q = torch.stack([table[c & 15], table[c >> 4]], dim=2)
    if fmt == "nvfp4":
        a = t["block_scales"].view(torch.float8_e4m3fn).to(torch.float32)
    else:
        a = torch.exp2(t["block_scales"].to(torch.float64) - 127.0).to(torch.float32)
    return (q.view(rows, a.shape[1], -1) * a.unsqueeze(2)).view(rows, -1)


def _plain_matmul(x, w, fmt, dtype):
    y = _values(x, fmt) @ _values(w, fmt).t()
    if fmt == "nvfp4":
        y = (y.double() * (x["tensor_scale"].double() * w["tensor_scale"].double())).to(torch.float32)
    return y.to(dtype)


def _plain_norm(s, fmt):
    h = s["x"]
    if s["residual"] is not None:
        h = (h.to(torch.float32) + s["residual"].to(torch.float32)).to(h.dtype)
    v = h.double()
    r = 1.0 / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)
    return h, _quantize(v * (s["weight"].double() * s["b"].double()) * r, fmt)


def _plain_glu(gate_up, b, fmt):
    gate, up = gate_up.double().chunk(2, dim=1)
    return _quantize(gate / (1.0 + torch.exp(-gate)) * up * b.double(), fmt)


# ---------------------------------------------------------------------------
# Inputs

def _activations(gen, tokens, cols, dtype):
    """N(0, 1) with one channel in a hundred 20 times as large, as hidden states have them."""
    x = torch.randn(tokens, cols, generator=gen, device="cuda")
    at = torch.randperm(cols, generator=gen, device="cuda")[:max(1, cols // 100)]
    x[:, at] *= 20.0
    return x.to(dtype)


def _col_scales(gen, cols):
    return torch.exp(0.3 * torch.randn(cols, generator=gen, device="cuda")).to(torch.bfloat16)


def _weights(gen, rows, b, fmt):
    """N(0, 0.02^2) with outlier columns, divided by the column scales and quantized."""
    w = torch.randn(rows, b.shape[0], generator=gen, device="cuda") * 0.02
    at = torch.randperm(b.shape[0], generator=gen, device="cuda")[:max(1, b.shape[0] // 200)]
    w[:, at] *= 15.0
    return _quantize(w.double() / b.double(), fmt)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    fmt, t, k, dtype = case["fmt"], case["tokens"], case["cols"], DTYPES[case["dtype"]]
    s = {"op": case["op"], "fmt": fmt, "dtype": dtype}
    b = _col_scales(gen, k)
    if case["op"] == "matmul":
        x = _activations(gen, t, k, torch.bfloat16)
        s.update(x=_quantize(x.double() * b.double(), fmt), w=_weights(gen, case["rows"], b, fmt))
    elif case["op"] == "glu":
        # gate and up side by side, as one product over the stacked gate and up weights gives them
        s.update(x=(2.0 * torch.randn(t, 2 * k, generator=gen, device="cuda")).to(dtype), b=b)
    else:
        s.update(x=_activations(gen, t, k, dtype), residual=None, b=b)
        if case["op"] == "mlp" or case["residual"]:
            s["residual"] = (4.0 * torch.randn(t, k, generator=gen, device="cuda")).to(dtype)
        s["weight"] = (1.0 + 0.2 * torch.randn(k, generator=gen, device="cuda")).to(dtype)
        if case["op"] == "mlp":
            s["b2"] = _col_scales(gen, case["inter"])
            s["w1"] = _weights(gen, 2 * case["inter"], b, fmt)
            s["w2"] = _weights(gen, k, s["b2"], fmt)
    return s


# ---------------------------------------------------------------------------
# One pass

def _returned(q):
    """MXFP8 codes and scales as the values they stand for."""
    return {"codes": q["codes"].view(torch.float8_e4m3fn), "block_scales": q["block_scales"].view(torch.float8_e8m0fnu)}


def run(state):
    s, op, fmt = state, state["op"], state["fmt"]
    if own:
        import calibration_free_weight_dualquant_b200 as dq
        if op == "matmul":
            return dq.dq_matmul(s["x"], s["w"], fmt, out_dtype=s["dtype"], check=False)
        if op == "glu":
            return _returned(dq.dq_glu_quant(s["x"], s["b"], fmt, check=False))
        q = dq.dq_norm_quant(s["x"], s["weight"], s["b"], fmt, residual=s["residual"], eps=EPS, check=False)
        if op == "norm":
            return {"h": q["residual"], **_returned(q)} if s["residual"] is not None else _returned(q)
        g = dq.dq_glu_quant(dq.dq_matmul(q, s["w1"], fmt, out_dtype=s["dtype"], check=False), s["b2"], fmt, check=False)
        return {"h": q["residual"], "y": dq.dq_matmul(g, s["w2"], fmt, out_dtype=s["dtype"], check=False)}
    if op == "matmul":
        return _plain_matmul(s["x"], s["w"], fmt, s["dtype"])
    if op == "glu":
        return _returned(_plain_glu(s["x"], s["b"], fmt))
    h, q = _plain_norm(s, fmt)
    if op == "norm":
        return {"h": h, **_returned(q)} if s["residual"] is not None else _returned(q)
    g = _plain_glu(_plain_matmul(q, s["w1"], fmt, s["dtype"]), s["b2"], fmt)
    return {"h": h, "y": _plain_matmul(g, s["w2"], fmt, s["dtype"])}


# ---------------------------------------------------------------------------
# The definitions in 64 bits, written apart from the plain form: grids as sorted tables, nearest entries by
# bisection between the entries' midpoints.

def _grid(fmt, device):
    if fmt == "mxfp8":
        g = [m / 512 for m in range(8)] + [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)][:-1]
    else:
        g = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    return torch.tensor(g, dtype=torch.float64, device=device)


def _nearest(v, grid):
    """Index of the entry nearest to each magnitude; a tie goes to the even index (the even mantissa)."""
    mid = (grid[1:] + grid[:-1]) / 2
    low = torch.bucketize(v, mid)               # a value on a midpoint: the lower entry
    high = torch.bucketize(v, mid, right=True)  # ... and the upper one
    return torch.where(low % 2 == 0, low, high)


def _exact_quantize(x, fmt):
    """(grid values with signs, block scales, tensor scale) in fp64."""
    n = GROUP[fmt]
    blocks = x.reshape(-1, n)
    top = blocks.abs().max(dim=1).values
    sT = 1.0
    if fmt == "nvfp4":
        sT = float((x.abs().max() / 2688).float()) or 1.0
        scales = _grid("mxfp8", x.device)
        a = scales[_nearest(top / 6 / sT, scales).clamp(min=1)]
    else:
        ratio = top / (448 if fmt == "mxfp8" else 6)
        down = torch.pow(2.0, torch.floor(torch.log2(ratio.clamp(min=2.0 ** -130))))
        a = torch.where(ratio - down >= 2 * down - ratio, 2 * down, down).clamp(2.0 ** -126, 2.0 ** 126)
    a = torch.where(top > 0, a, torch.ones_like(a))
    grid = _grid(fmt, x.device)
    q = grid[_nearest((blocks / (a * sT)[:, None]).abs(), grid)] * blocks.sign()
    return q.view(x.shape), a.view(x.shape[0], -1), sT


def _exact_decode(t, fmt):
    """Codes and scales to fp64 by their fields: sign, exponent, mantissa."""
    c = t["codes"].long()
    if fmt != "mxfp8":
        c = torch.stack((c % 16, c // 16), -1).flatten(1)
        e, m, top, width, bias = c // 2 % 4, c % 2, c // 8, 2.0, 1
    else:
        e, m, top, width, bias = c // 8 % 16, c % 8, c // 128, 8.0, 7
    q = torch.where(e > 0, (1 + m / width) * torch.pow(2.0, (e - bias).double()), m / width * 2.0 ** (1 - bias))
    q = q * (1 - 2 * top)
    s = t["block_scales"].long()
    if fmt == "nvfp4":
        a = torch.where(s > 7, (1 + s % 8 / 8.0) * torch.pow(2.0, (s // 8 - 7).double()), s / 512.0)
    else:
        a = torch.pow(2.0, (s - 127).double())
    return q, a, float(t["tensor_scale"])


def _scaled(q, a, sT):
    return (q.view(a.shape[0], a.shape[1], -1) * (a * sT)[:, :, None]).flatten(1)


def _exact_norm(s):
    h = s["x"].double()
    if s["residual"] is not None:
        h = (h + s["residual"].double()).to(s["dtype"]).double()  # the sum as the residual stream keeps it
    return h, h / (h.square().sum(1, keepdim=True) / h.shape[1] + EPS).sqrt() * s["weight"].double() * s["b"].double()


def exact(case, seed):
    s = prepare(case, seed)
    fmt, op = s["fmt"], s["op"]
    if op == "matmul":
        return _scaled(*_exact_decode(s["x"], fmt)) @ _scaled(*_exact_decode(s["w"], fmt)).T

    def silu_mul(gu, b):
        n = gu.shape[1] // 2
        return torch.sigmoid(gu[:, :n]) * gu[:, :n] * gu[:, n:] * b.double()

    if op == "glu":
        q, a, _ = _exact_quantize(silu_mul(s["x"].double(), s["b"]), fmt)
        return {"codes": q, "block_scales": a}
    h, y = _exact_norm(s)
    if op == "norm":
        q, a, _ = _exact_quantize(y, fmt)
        return {"h": h, "codes": q, "block_scales": a} if s["residual"] is not None else {"codes": q, "block_scales": a}
    gu = _scaled(*_exact_quantize(y, fmt)) @ _scaled(*_exact_decode(s["w1"], fmt)).T
    gu = gu.to(s["dtype"]).double()  # the product's output as the glu reads it
    return {"h": h, "y": _scaled(*_exact_quantize(silu_mul(gu, s["b2"]), fmt)) @ _scaled(*_exact_decode(s["w2"], fmt)).T}
