"""The operators of a quantised transformer MLP on real sizes: what each one is given, its plain form,
its calls in this package, and its value in 64 bits.

Four kinds of case ("op"):

  norm      h = x + residual, y = h / rms(h) * weight, codes and one scale a row (capi.rmsnorm_q8_run)
  act       y = silu(gate) * up, codes and one scale a row               (capi.silu_mul_q8_run)
  linear    y[m,n] = scale_x[m] * scale_w[n] * sum_k x[m,k] * w[n,k] + bias[n]  (q8.LinearQ8)
  normlin   the first into the third, as a layer's first product takes it

Codes are int8 ("i8") or e4m3 ("e4m3"); a row's scale is the amax of its values over 127 or 448 (1 for
a row of zeros), a code is the value over the scale, rounded to nearest even. Sums are in 32 bits.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
TOP = {"i8": 127.0, "e4m3": 448.0}
EPS = 1e-6
MOST_FLOPS = 2.0 * 8192 * 4096 * 8192  # of a drawn case: the largest listed one's
MOST_VALUES = 4096 * 16384


def listed():
    return [
        # one token of a running sequence: latency
        {"name": "norm 1 x 4096", "op": "norm", "rows": 1, "cols": 4096, "type": "bf16",
         "codes": "e4m3", "residual": True},
        # a prompt's tokens: bandwidth
        {"name": "norm 8192 x 4096", "op": "norm", "rows": 8192, "cols": 4096, "type": "bf16",
         "codes": "e4m3", "residual": True},
        # a ragged batch of a model whose width is no power of two, in 32 bits, no residual
        {"name": "norm 1501 x 5001 f32", "op": "norm", "rows": 1501, "cols": 5001, "type": "f32",
         "codes": "e4m3", "residual": False},
        # eight sequences, one token each, between the two products of the MLP
        {"name": "act 8 x 8192", "op": "act", "rows": 8, "cols": 8192, "type": "bf16",
         "codes": "e4m3"},
        # a prompt's tokens at the MLP's inner width
        {"name": "act 4096 x 16384", "op": "act", "rows": 4096, "cols": 16384, "type": "bf16",
         "codes": "e4m3"},
        # one token: the weights' bytes are all there is
        {"name": "linear i8 1 x 4096 x 4096", "op": "linear", "rows": 1, "n": 4096, "k": 4096,
         "codes": "i8", "type": "bf16", "bias": False},
        # a batch of running sequences
        {"name": "linear i8 64 x 8192 x 4096", "op": "linear", "rows": 64, "n": 8192, "k": 4096,
         "codes": "i8", "type": "bf16", "bias": False},
        # a prompt of a small model with odd widths, a bias, sums kept in 32 bits
        {"name": "linear i8 777 x 2500 x 1001", "op": "linear", "rows": 777, "n": 2500, "k": 1001,
         "codes": "i8", "type": "f32", "bias": True},
        # a long prompt: the rate of the tensor cores
        {"name": "linear i8 8192 x 4096 x 8192", "op": "linear", "rows": 8192, "n": 4096,
         "k": 8192, "codes": "i8", "type": "bf16", "bias": False},
        # sixteen sequences, e4m3 weights
        {"name": "linear e4m3 16 x 4096 x 8192", "op": "linear", "rows": 16, "n": 4096, "k": 8192,
         "codes": "e4m3", "type": "f16", "bias": True},
        # a prompt, e4m3
        {"name": "linear e4m3 4096 x 8192 x 4096", "op": "linear", "rows": 4096, "n": 8192,
         "k": 4096, "codes": "e4m3", "type": "bf16", "bias": False},
        # a short prompt's residual, norm and first product, int8
        {"name": "normlin i8 256 x 6144 x 4096", "op": "normlin", "rows": 256, "n": 6144,
         "k": 4096, "codes": "i8", "type": "bf16", "residual": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "act", "linear", "linear", "linear", "normlin"])
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    rows = _log(rng, 1, 8192)
    if op in ("norm", "act"):
        cols = _log(rng, 256, 16384)
        if rng.random() < 0.7:  # the widths of most models; the others are odd
            cols = -(-cols // 128) * 128
        rows = max(1, min(rows, MOST_VALUES // (cols * (2 if kind == "f32" else 1))))
        case = {"op": op, "rows": rows, "cols": cols, "type": kind, "codes": "e4m3"}
        if op == "norm":
            case["residual"] = rng.random() < 0.7
        return case
    n, k = _log(rng, 200, 16384), _log(rng, 200, 16384)
    if rng.random() < 0.7:
        n, k = -(-n // 128) * 128, -(-k // 128) * 128
    rows = max(1, min(rows, int(MOST_FLOPS / (2.0 * n * k)), MOST_VALUES // max(n, k)))
    case = {"op": op, "rows": rows, "n": n, "k": k, "type": kind}
    if op == "linear":
        case.update(codes=rng.choice(["i8", "i8", "e4m3"]), bias=rng.random() < 0.4)
    else:
        case.update(codes="i8", residual=rng.random() < 0.7)
    return case


# ------------------------------------------------------------------------------------- inputs
def _activations(gen, rows, cols, dtype):
    """Normal values, a few channels of which are large, as a transformer's hidden states have them."""
    v = torch.randn(rows, cols, generator=gen, device=DEV)
    loud = torch.rand(cols, generator=gen, device=DEV) < 0.005
    v = torch.where(loud, v * 12.0, v)
    return v.to(dtype)


def _padded(rows, cols, dtype):
    """A [rows, cols] view whose row pitch is a multiple of 16 bytes."""
    size = torch.empty(0, dtype=dtype).element_size()
    pitch = -(-cols * size // 16) * 16 // size
    return torch.empty(rows, pitch, dtype=dtype, device=DEV)[:, :cols]


def _codes(v, codes):
    """Rows of values as codes in padded rows, and their scales."""
    amax = v.abs().amax(dim=1)
    scale = torch.where(amax > 0, amax / TOP[codes], torch.ones_like(amax))
    out = _padded(*v.shape, torch.int8 if codes == "i8" else torch.float8_e4m3fn)
    v = v / scale[:, None]
    out.copy_(v.round() if codes == "i8" else v)
    return out, scale


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op, rows, dtype = case["op"], case["rows"], TYPES[case["type"]]
    code_type = torch.int8 if case["codes"] == "i8" else torch.float8_e4m3fn
    s = {"case": case}
    if op in ("norm", "normlin"):
        cols = case["cols"] if op == "norm" else case["k"]
        s["x"] = _activations(gen, rows, cols, dtype)
        s["weight"] = (1.0 + 0.1 * torch.randn(cols, generator=gen, device=DEV)).to(dtype)
        s["residual"] = _activations(gen, rows, cols, dtype) if case["residual"] else None
        s["residual_out"] = torch.empty_like(s["x"]) if case["residual"] else None
        s["q"] = _padded(rows, cols, code_type)
        s["scale"] = torch.empty(rows, dtype=torch.float32, device=DEV)
    if op == "act":
        both = _activations(gen, rows, 2 * case["cols"], dtype)  # as one product leaves the two
        s["gate"], s["up"] = both[:, :case["cols"]], both[:, case["cols"]:]
        s["q"] = _padded(rows, case["cols"], code_type)
        s["scale"] = torch.empty(rows, dtype=torch.float32, device=DEV)
    if op in ("linear", "normlin"):
        n, k = case["n"], case["k"]
        if op == "linear":
            s["x"], s["scale_x"] = _codes(_activations(gen, rows, k, torch.float32), case["codes"])
        w = torch.randn(n, k, generator=gen, device=DEV) / math.sqrt(k)
        s["w"], s["scale_w"] = _codes(w, case["codes"])
        s["bias"] = None
        if case.get("bias"):
            s["bias"] = torch.randn(n, generator=gen, device=DEV)
        s["y"] = torch.empty(rows, n, dtype=dtype, device=DEV)
        if own:
            from fp8_implicit_gemm_gb300 import q8
            s["linear"] = q8.LinearQ8(s["w"], s["scale_w"], bias=s["bias"], max_rows=rows)
    return s


# ------------------------------------------------------------------------------------- one pass
def _plain_quantise(y, codes):
    amax = y.abs().amax(dim=1)
    scale = torch.where(amax > 0, amax / TOP[codes], torch.ones_like(amax))
    v = y / scale[:, None]
    if codes == "i8":
        return v.round().clamp(-127.0, 127.0).to(torch.int8), scale
    return v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scale


def _plain_norm(s):
    h = s["x"].float()
    out = None
    if s["residual"] is not None:
        h = h + s["residual"].float()
        out = h.to(s["x"].dtype)
    y = h * torch.rsqrt(h.square().mean(dim=1, keepdim=True) + EPS) * s["weight"].float()
    q, scale = _plain_quantise(y, s["case"]["codes"])
    return q, scale, out


def _plain_linear(s, x, scale_x):
    y = x.float() @ s["w"].float().t()
    y = y * scale_x[:, None] * s["scale_w"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(s["y"].dtype)


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        from fp8_implicit_gemm_gb300 import capi
        if op in ("norm", "normlin"):
            capi.rmsnorm_q8_run(s["x"], s["weight"], s["q"], s["scale"], EPS,
                                residual=s["residual"], residual_out=s["residual_out"])
            if op == "norm":
                return _norm_outputs(s["q"], s["scale"], s["residual_out"])
            s["linear"](s["q"], s["scale"], s["y"])
            return _normlin_outputs(s["y"], s["scale"], s["residual_out"])
        if op == "act":
            capi.silu_mul_q8_run(s["gate"], s["up"], s["q"], s["scale"])
            return {"q": s["q"], "scale": s["scale"]}
        s["linear"](s["x"], s["scale_x"], s["y"])
        return {"y": s["y"]}
    if op in ("norm", "normlin"):
        q, scale, out = _plain_norm(s)
        if op == "norm":
            return _norm_outputs(q, scale, out)
        return _normlin_outputs(_plain_linear(s, q, scale), scale, out)
    if op == "act":
        g, u = s["gate"].float(), s["up"].float()
        q, scale = _plain_quantise(g / (1.0 + torch.exp(-g)) * u, s["case"]["codes"])
        return {"q": q, "scale": scale}
    return {"y": _plain_linear(s, s["x"], s["scale_x"])}


def _norm_outputs(q, scale, out):
    r = {"q": q, "scale": scale}
    if out is not None:
        r["residual_out"] = out
    return r


def _normlin_outputs(y, scale, out):
    r = {"y": y, "scale": scale}
    if out is not None:
        r["residual_out"] = out
    return r


# ------------------------------------------------------------------------------------- 64 bits
def _exact_e4m3(v):
    """v rounded to the nearest e4m3 value, ties to the even one: three bits behind the first, the
    smallest step 2^-9, the largest value 448."""
    mag = v.abs()
    power = torch.floor(torch.log2(mag.clamp(min=2.0 ** -6)))
    power = torch.where(torch.exp2(power) > mag.clamp(min=2.0 ** -6), power - 1, power)
    power = torch.where(torch.exp2(power + 1) <= mag, power + 1, power)
    step = torch.exp2(power - 3)
    return torch.sign(v) * torch.clamp(torch.round(mag / step) * step, max=448.0)


def _exact_codes(y, codes):
    scale = y.abs().max(dim=1).values / TOP[codes]
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    v = y / scale.unsqueeze(1)
    return torch.round(v) if codes == "i8" else _exact_e4m3(v), scale


def exact(case, seed):
    s = prepare(case, seed)
    op, codes = case["op"], case["codes"]
    found = {}
    if op in ("norm", "normlin"):
        h = s["x"].double()
        if s["residual"] is not None:
            h += s["residual"].double()
            found["residual_out"] = h.clone()
        rms = torch.sqrt(torch.sum(h * h, dim=1) / h.shape[1] + EPS)
        q, found["scale"] = _exact_codes(h / rms.unsqueeze(1) * s["weight"].double(), codes)
        if op == "norm":
            found["q"] = q
            return found
        x, scale_x = q, found["scale"]
    elif op == "act":
        g = s["gate"].double()
        q, scale = _exact_codes(g * torch.sigmoid(g) * s["up"].double(), codes)
        return {"q": q, "scale": scale}
    else:
        x, scale_x = s["x"].double(), s["scale_x"].double()
    y = torch.mm(x, s["w"].double().t()) * torch.outer(scale_x, s["scale_w"].double())
    if s["bias"] is not None:
        y += s["bias"].double()
    found["y"] = y
    return found


# ------------------------------------------------------------------------------------- work
def work(case):
    """Each input read once, each output written once; the multiplications and additions."""
    op, rows, size = case["op"], case["rows"], BYTES[case["type"]]
    nbytes = flops = 0.0
    if op in ("norm", "normlin"):
        cols = case["cols"] if op == "norm" else case["k"]
        nbytes += rows * cols * size * (3 if case["residual"] else 1) + cols * size + 4 * rows
        flops += 7.0 * rows * cols
        if op == "norm":
            nbytes += rows * cols
    if op == "act":
        nbytes += rows * case["cols"] * (2 * size + 1) + 4 * rows
        flops += 8.0 * rows * case["cols"]
    if op in ("linear", "normlin"):
        n, k = case["n"], case["k"]
        nbytes += n * k + 4 * n + rows * n * size
        if op == "linear":
            nbytes += rows * k + 4 * rows + (4 * n if case["bias"] else 0)
        flops += 2.0 * rows * n * k
    return {"bytes": nbytes, "flops": flops}
