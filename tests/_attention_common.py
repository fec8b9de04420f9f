"""Plain 64-bit forms of the attention operators, and the bounds the kernels are held to.

Written from the formulas in include/q8_attention.h, on torch float64 tensors, without the package's code.

Where the bounds come from (u = 2^-24, fp32's unit roundoff):
  * a normed head: a sum of at most 256 squares in at most 13 sequential additions errs by 14u at most, its
    root's reciprocal by half of that and 2^-22, three products and a division by u each: under 2^-20;
  * a turned pair (a, b): the angle's fraction of a turn, rounded to fp32, is off by 2^-25 turns, which is
    2^-22.3; sine and cosine err by 2 units of their last place (2^-23) each, the products and the sum by u each:
    under (|a| + |b|) * 2^-20.5 on top, under (|a| + |b|) * 2^-19 with the norm;
  * a score: one instruction of the tensor cores errs by at most 33 * 2^-25 + 2^-23 of the largest operand, and
    dim / 16 of them follow each other, so (dim / 16 + 1) * 2^-19.5 of sum |q k|; cached scales and the
    logarithm's base add 8u of it; a q in f16 is exact but for elements below 2^-14 of the row's largest, which
    err by 2^-25 of that: 2^-11 of sum max|q| |k| at most in all, far less as they are few, so
    dim * 2^-25 * max|q| max|k|. Off by d, a score takes its weight off by a factor of e^d, and the sum of the
    weights too: 2d of sum p |v| (for d small);
  * a weight is rounded to f16 (cache) or to the value type (prompt) before it meets v, 2^-11 or half a step of the
    type; exp2 errs by 2^-22; the sums over keys by (keys / 16 + 1) * 2^-23 of sum p |v| (each addition cut below
    its last bit) and as much over again for the joins: 2^-9 * 2^-14 * keys;
  * the output's own rounding.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24
ROUND = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}
TOP = {"i8": 127.0, "e4m3": 448.0}
CODES = ["i8", "e4m3", "i4"]
CODE_DTYPE = {"i8": torch.int8, "e4m3": torch.float8_e4m3fn, "i4": torch.uint8}
CODE_ARG = {"i8": torch.int8, "e4m3": torch.float8_e4m3fn, "i4": 4}


def randn(*shape, dtype=torch.float32, seed=0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=device).to(dtype)


def heads64(x, weight=None, eps=1e-6, freqs=None, axis=None, positions=None, rot=0, adjacent=False):
    """The normed and turned heads, and what their error is measured by (|a| + |b| of a turned element)."""
    y = x.double().clone()
    if weight is not None:
        mean = (y * y).sum(dim=-1, keepdim=True) / y.shape[-1] + eps
        y = torch.where(mean == 0, torch.zeros_like(y), y / torch.sqrt(mean)) * weight.double()
    size = y.abs()
    if rot:
        angle = positions.double()[axis].t() * freqs  # [tokens, pairs]
        c, s = angle.cos()[:, None], angle.sin()[:, None]
        first = slice(0, rot, 2) if adjacent else slice(0, rot // 2)
        second = slice(1, rot, 2) if adjacent else slice(rot // 2, rot)
        a, b = y[..., first].clone(), y[..., second].clone()
        y[..., first], y[..., second] = a * c - b * s, b * c + a * s
        both = a.abs() + b.abs()
        size[..., first], size[..., second] = both, both
    return y, size


def codes64(v, codes):
    """(codes as float64, scale, lowest) of finite rows, from their values."""
    v = v.double()
    if codes == "i4":
        lowest, highest = v.amin(-1, keepdim=True), v.amax(-1, keepdim=True)
        width = (highest - lowest)
        flat = width == 0
        q = torch.round(15.0 * (v - lowest) / torch.where(flat, torch.ones_like(width), width))
        return q, torch.where(flat, torch.ones_like(width), width / 15.0)[..., 0], lowest[..., 0]
    amax = v.abs().amax(-1, keepdim=True)
    flat = amax == 0
    q = TOP[codes] * v / torch.where(flat, torch.ones_like(amax), amax)
    if codes == "i8":
        q = torch.round(q)
    else:
        _, power = torch.frexp(q.abs().clamp(min=2.0 ** -6))
        step = torch.exp2(power.double() - 4)
        q = torch.round(q / step) * step
    return q, torch.where(flat, torch.ones_like(amax), amax / TOP[codes])[..., 0], None


def unpack(q, codes):
    """Codes of a cache as float64."""
    if codes == "i4":
        b = q.to(torch.int64)
        return torch.stack([b & 15, b >> 4], dim=-1).flatten(-2).double()
    return q.to(torch.float32).double()


def values64(cache, name, codes):
    """All values of a cache, [pages, kv_heads, page_size, dim]."""
    q, scale = unpack(getattr(cache, name + "_codes"), codes), getattr(cache, name + "_scale").double()
    return q * scale[..., :1] + scale[..., 1:] if codes == "i4" else q * scale[..., None]


def fill_cache(cache, codes, seed, spread=1.0):
    """Random keys and values in every page, by the formulas (not the kernels)."""
    for i, name in enumerate("kv"):
        shape = cache.k_codes.shape[:3] + (cache.head_dim,)
        v = randn(*shape, seed=seed + i) * spread
        q, scale, lowest = codes64(v, codes)
        if codes == "i4":
            b = q.to(torch.uint8)
            getattr(cache, name + "_codes").copy_(b[..., 0::2] | (b[..., 1::2] << 4))
            getattr(cache, name + "_scale").copy_(torch.stack([scale, lowest], dim=-1))
        else:
            getattr(cache, name + "_codes").copy_(q.to(CODE_DTYPE[codes]))
            getattr(cache, name + "_scale").copy_(scale)


def attention64(q, k, v, limits, scale):
    """One sequence: q [rows, heads, dim], k and v [keys, kv_heads, dim], row i sees limits[i] keys. Gives o, sum p|v|
    and the largest error of a score."""
    rows, heads, dim = q.shape
    keys, kv = k.shape[:2]
    q = q.double().view(rows, kv, heads // kv, dim)
    k, v = k.double(), v.double()
    x = torch.einsum("rhgd,khd->rhgk", q, k) * scale
    mag = torch.einsum("rhgd,khd->rhgk", q.abs(), k.abs()) * abs(scale)
    seen = (torch.arange(keys, device=q.device) < limits[:, None])[:, None, None]
    x = x.masked_fill(~seen, -torch.inf)
    p = torch.softmax(x, dim=-1) if keys else x
    p = torch.where((limits > 0)[:, None, None, None], p, torch.zeros_like(p))
    vs = torch.where(seen.any(dim=0)[0, 0][:, None, None], v, torch.zeros_like(v))  # what no row sees
    o = torch.einsum("rhgk,khd->rhgd", p, vs).reshape(rows, heads, dim)
    size = torch.einsum("rhgk,khd->rhgd", p, vs.abs()).reshape(rows, heads, dim)
    worst = 0.0
    if keys and rows:
        top = float((mag * seen).max())
        worst = ((dim / 16 + 1) * 2.0 ** -19.5 + 8 * U) * top
        worst += dim * 2.0 ** -25 * float(q.abs().max() * k.abs().max()) * abs(scale)
    return o, size, worst


def check_attention(got, want, size, worst, weight_round, keys, what=""):
    r, tiny = ROUND[got.dtype], TINY[got.dtype]
    err = (2.1 * worst + weight_round + 2.0 ** -21 + keys * 2.0 ** -23) * size
    bound = (err + (want.abs() + err) * r) * (1 + 2.0 ** -20) + tiny
    assert bool(torch.isfinite(got).all()), f"{what}: not finite"
    off = (got.double() - want).abs() - bound
    assert off.numel() == 0 or float(off.max()) <= 0.0, f"{what}: {float(off.max()):.3g} past its bound"
