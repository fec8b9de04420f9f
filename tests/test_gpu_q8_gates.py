"""The gated activation over the whole range of gates, against its formula in 64 bits.

The bound of a value y = silu(g) * u, relative (u = 2^-24): exp's argument is scaled by log2(e) in fp32 and
the result approximated to 2 ulp, (|g| + 4) * 2u; the sum, the reciprocal and the products by under
16u; and below -87.3 the exponential is a subnormal number, a multiple of 2^-149, of which two may be
lost: 2^-148 / exp(g)."""
import pytest
import torch

from fp8_implicit_gemm_gb300 import capi
from _q8_common import CODE_TYPES, TOP, U, VALUE_TYPES, act64, check_codes

pytestmark = pytest.mark.gpu


def value_err(gate):
    g = gate.double()
    return (g.abs() + 4) * 2 * U + 16 * U + torch.where(g < -87.0, 2.0 ** -148 / torch.exp(g), 0.0)


@pytest.mark.parametrize("lo,hi,up", [(-89.0, -87.0, 1e30), (-95.0, -89.0, 1e30), (-87.0, -80.0, 1.0),
                                      (-80.5, -79.5, 1.0), (-80.0, 0.0, 3.0), (0.0, 80.0, 3.0),
                                      (79.5, 89.0, 1.0)])
def test_values(lo, hi, up):
    """Rows of one column: the scale is the value's magnitude over the type's largest code."""
    gate = torch.linspace(lo, hi, 20011, device="cuda")[:, None].contiguous()
    up = torch.full_like(gate, up)
    for code_dtype in CODE_TYPES:
        q = torch.empty(gate.shape, dtype=code_dtype, device="cuda")
        scale = torch.empty(gate.shape[0], device="cuda")
        capi.silu_mul_q8_run(gate, up, q, scale)
        y = act64(gate, up)[:, 0]
        want = y.abs() / TOP[code_dtype]
        keep = want > 2.0 ** -126  # a scale below that is rounded coarsely itself
        off = (scale.double() - want).abs() / want - value_err(gate[:, 0])
        assert float(keep.double().mean()) > 0.8 and float(off[keep].max()) <= 0.0
        assert torch.equal(q[:, 0].float()[keep], (torch.sign(y) * TOP[code_dtype]).float()[keep])


@pytest.mark.parametrize("cols,offset", [(8, 0), (1000, 0), (4096, 0), (1001, 1), (4098, 2),
                                         (12501, 1), (12502, 2), (32768, 0)])
@pytest.mark.parametrize("dtype", VALUE_TYPES)
def test_codes(dtype, cols, offset):
    """Whole rows of gates between -89 and -87, and rows with one of them among ordinary ones, in
    every kernel: whole 16-byte chunks, pairs and single elements, in registers and in shared memory."""
    g = torch.Generator(device="cuda").manual_seed(cols)
    pitch = -(-cols // 16) * 16 + offset
    gate, up = (torch.empty(4, pitch, dtype=dtype, device="cuda")[:, :cols] for _ in range(2))
    gate.copy_(torch.randn(4, cols, generator=g, device="cuda") * 3)
    up.copy_(torch.randn(4, cols, generator=g, device="cuda") + 3)
    gate[0] = (torch.rand(cols, generator=g, device="cuda") * 2 - 89).to(dtype)
    gate[1, cols // 2] = -88.0
    gate[2] = -88.0
    up[:, 0] = 1.0
    if dtype != torch.float16:  # whose up has no room for it
        up[0] *= 2.0 ** 100
        up[2] *= 2.0 ** 100
    for code_dtype in CODE_TYPES:
        q = torch.empty(4, cols, dtype=code_dtype, device="cuda")
        scale = torch.empty(4, device="cuda")
        capi.silu_mul_q8_run(gate, up, q, scale)
        y = act64(gate, up)
        for row in range(4):
            err = float(value_err(gate[row]).max())
            if dtype == torch.float16 and row in (0, 2):  # values near fp32's smallest normal number
                err += 2.0 ** -148 / float(y[row].abs().amax()) * TOP[code_dtype]
            check_codes(q[row:row + 1], scale[row:row + 1], y[row:row + 1], 2 * err, err, f"row {row}")


def test_far_gates_of_either_sign():
    gate = torch.tensor([[-1e30, -300.0, -104.5, 100.0, 300.0, 2e38, 3e38, 0.0]], device="cuda")
    up = torch.tensor([[1e30, 1e30, 1.0, 1e-30, 1e-30, 1e-30, 1e-38, 1e30]], device="cuda")
    q, scale = torch.empty(1, 8, dtype=torch.int8, device="cuda"), torch.empty(1, device="cuda")
    capi.silu_mul_q8_run(gate, up, q, scale)
    assert float(scale[0]) == pytest.approx(2e8 / 127, rel=1e-6)
    assert q[0].tolist() == [0, 0, 0, 0, 0, 127, 0, 0]


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_gates_that_are_not_finite_mark_their_row(bad):
    """As any row with such values is: silu(-inf) is -inf * 0."""
    for cols in (8, 1001, 4096, 12501):
        g = torch.Generator(device="cuda").manual_seed(cols)
        gate = torch.randn(3, cols, generator=g, device="cuda")
        up = torch.randn(3, cols, generator=g, device="cuda")
        a = torch.empty(3, cols, dtype=torch.int8, device="cuda"), torch.empty(3, device="cuda")
        b = torch.empty_like(a[0]), torch.empty_like(a[1])
        capi.silu_mul_q8_run(gate, up, *a)
        gate[1, cols - 1] = bad
        capi.silu_mul_q8_run(gate, up, *b)
        assert bool(torch.isnan(b[1][1])) and int(b[0][1].abs().max()) == 0
        for row in (0, 2):
            assert torch.equal(a[0][row], b[0][row]) and torch.equal(a[1][row], b[1][row])
