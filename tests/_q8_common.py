"""Plain 64-bit forms of the 8-bit transformer operators, and the bounds the kernels are held to.

Written from the formulas in include/q8.h, on torch float64 tensors, without the package's code.

Where the bounds come from (u = 2^-24, fp32's unit roundoff):
  * scale of a norm: amax and the weight's product err by 2u each, the root of the mean square by
    half of what a sum of n positive terms in any order of at most 160 sequential additions errs
    (80u), the square root, the division and two products by 2u each: under 2^-17;
  * scale of an activation: silu's exponential errs by (|g| + 4) * 2u at most (its argument is
    scaled by log2(e) in fp32, and the result approximated to 2 ulp), the rest by under 16u;
  * a code: the quotient v / s errs by what v errs, its own row's amax errs and a division and a
    product err: 16u of it for a norm (its root cancels), and the code is then the nearest one, so
    it lies within half a step of the quotient, and that much more;
  * an integer product of K <= 1024 codes is exact, so only the scaling (two products), the bias's
    addition and the type's rounding err;
  * a tensor-core sum of floating-point products: an instruction adds at most 32 products and the
    accumulator aligned to the largest, cut 2 bits below its last bit: 33 * 2^-25 + 2^-23 of the
    largest operand, which sum(|x * w|) bounds: (K / 16 + 1) * 2^-19.5 of that sum in all, more
    than any order of plain fp32 additions of as many terms errs in K / 16 instructions of 16.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24
ROUND = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}
TOP = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}
VALUE_TYPES = [torch.bfloat16, torch.float16, torch.float32]
CODE_TYPES = [torch.int8, torch.float8_e4m3fn]


def padded(rows, cols, dtype, extra=0, device="cuda"):
    """[rows, cols] with a pitch of whole 16-byte units, `extra` such units more than it needs."""
    size = torch.empty(0, dtype=dtype).element_size()
    unit = 16 // size
    pitch = (-(-cols // unit) + extra) * unit
    return torch.empty(rows, pitch, dtype=dtype, device=device)[:, :cols]


def norm64(x, weight, eps, residual=None):
    h = x.double()
    if residual is not None:
        h = h + residual.double()
    return h, h / torch.sqrt((h * h).sum(dim=1, keepdim=True) / h.shape[1] + eps) * weight.double()


def act64(gate, up):
    g = gate.double()
    return g / (1.0 + torch.exp(-g)) * up.double()


def linear64(x, scale_x, w, scale_w, bias=None):
    """y and sum(|x * w|) scaled, both in 64 bits."""
    xs, ws = x.to(torch.float32).double(), w.to(torch.float32).double()
    s = scale_x.double()[:, None] * scale_w.double()[None, :]
    y, mag = (xs @ ws.t()) * s, (xs.abs() @ ws.abs().t()) * s.abs()
    if bias is not None:
        y = y + bias.double()
        mag = mag + bias.double().abs()
    return y, mag


def scale64(y, code_dtype):
    amax = y.abs().amax(dim=1)
    return torch.where(amax > 0, amax / TOP[code_dtype], torch.ones_like(amax))


def half_step(t, code_dtype):
    """Half the distance between the codes around t."""
    if code_dtype == torch.int8:
        return torch.full_like(t, 0.5)
    power = torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6)))
    return torch.exp2(power - 4)


def check_codes(q, scale, y, value_err, scale_err, what=""):
    """Codes and scales of the rows y (64 bits); value_err, scale_err: relative error bounds of a
    quotient and of a scale."""
    want = scale64(y, q.dtype)
    d = (scale.double() - want).abs()
    assert bool((d <= scale_err * want + 2.0 ** -148).all()), \
        f"{what}: scale off by {float((d / want).max()):.3g}, {scale_err:.3g} allowed"
    t = y / want[:, None]
    code = q.to(torch.float32).double()
    top = TOP[q.dtype]
    assert bool((code.abs() <= top).all()), what
    # a quotient just past a binade's end may round with the next binade's step
    bound = torch.maximum(half_step(t, q.dtype), half_step(t * (1 + value_err), q.dtype))
    off = (code - t).abs() - (bound + value_err * top)
    assert float(off.max()) <= 0.0, f"{what}: a code is {float(off.max()):.3g} past its bound"


def check_values(got, want, err, what=""):
    """got (a rounded type) against want (64 bits) whose fp32 computation errs by at most err."""
    r, tiny = ROUND[got.dtype], TINY[got.dtype]
    bound = (err + (want.abs() + err) * r) * (1 + 2.0 ** -20) + tiny
    off = (got.double() - want).abs() - bound
    assert not bool(torch.isnan(got).any()), f"{what}: NaN"
    assert float(off.max()) <= 0.0, f"{what}: {float(off.max()):.3g} past its bound"


def linear_err(mag, K, code_dtype):
    scaling = 6 * U * mag
    if code_dtype == torch.int8 and K <= 1024:
        return scaling
    return scaling + (K / 16 + 1) * 2.0 ** -19.5 * mag
