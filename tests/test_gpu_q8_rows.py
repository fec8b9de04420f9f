"""The norm and the gated activation with 8-bit outputs, against 64-bit forms of their formulas."""
import pytest
import torch

from fp8_implicit_gemm_gb300 import capi
from _q8_common import (CODE_TYPES, ROUND, TINY, U, VALUE_TYPES, act64, check_codes, check_values,
                        norm64, padded)

pytestmark = pytest.mark.gpu
EPS = 1e-6
# one token to many, one column to the widest row, widths around every vector and block size
SIZES = [(1, 1), (1, 7), (3, 8), (2, 31), (5, 64), (4, 127), (1, 256), (7, 257), (33, 1000),
         (2, 2048), (1, 4096), (300, 4096), (9, 5001), (5, 8192), (3, 11008), (2, 16384), (1, 16400),
         (4, 32760), (2, 32768)]
CODE_ERR = 16 * U


def values(rows, cols, dtype, seed, pitch_extra=0, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = padded(rows, cols, dtype, pitch_extra)
    out.copy_(torch.randn(rows, cols, generator=g, device="cuda") * spread)
    return out


def outputs(rows, cols, code_dtype, fill=0x55):
    q = torch.full((rows, cols + 32), fill, dtype=torch.uint8, device="cuda").view(code_dtype)
    return q[:, 16:16 + cols], torch.full((rows,), -1.0, device="cuda"), q


def check_guard(full, cols, fill=0x55):
    b = full.view(torch.uint8)
    assert bool((b[:, :16] == fill).all()) and bool((b[:, 16 + cols:] == fill).all())


def run_norm(x, weight, code_dtype, residual=None, eps=EPS):
    q, scale, full = outputs(*x.shape, code_dtype)
    out = None
    if residual is not None:
        out = torch.full((x.shape[0], x.shape[1] + 8), 7.0, dtype=x.dtype, device="cuda")
        capi.rmsnorm_q8_run(x, weight, q, scale, eps, residual=residual,
                            residual_out=out[:, :x.shape[1]])
        assert bool((out[:, x.shape[1]:] == 7.0).all())
        out = out[:, :x.shape[1]]
    else:
        capi.rmsnorm_q8_run(x, weight, q, scale, eps)
    torch.cuda.synchronize()
    check_guard(full, x.shape[1])
    return q, scale, out


@pytest.mark.parametrize("code_dtype", CODE_TYPES)
@pytest.mark.parametrize("dtype", VALUE_TYPES)
def test_norm_sizes(dtype, code_dtype):
    for i, (rows, cols) in enumerate(SIZES):
        x = values(rows, cols, dtype, 100 + i, pitch_extra=i % 3)
        weight = values(1, cols, dtype if i % 2 else torch.float32, 200 + i)[0] * 0.1 + 1.0
        residual = values(rows, cols, dtype, 300 + i, pitch_extra=i % 2) if i % 3 else None
        q, scale, out = run_norm(x, weight, code_dtype, residual)
        h, y = norm64(x, weight, EPS, residual)
        check_codes(q, scale, y, CODE_ERR, 2.0 ** -17, f"{rows}x{cols}")
        if residual is not None:
            check_values(out, h, h.abs() * U, f"{rows}x{cols} residual")


@pytest.mark.parametrize("offset", [1, 2, 3, 5])
def test_norm_any_alignment(offset):
    """Rows that start at any element: no vector access may assume a 16-byte boundary."""
    for dtype in VALUE_TYPES:
        base = values(6, 1100, dtype, 9)
        x, residual = base[:, offset:offset + 1031], base[:, 2 * offset:2 * offset + 1031]
        weight = values(1, 1040, dtype, 10)[0, offset:offset + 1031]
        buf = torch.zeros(6, 1100, dtype=dtype, device="cuda")
        out = buf[:, offset:offset + 1031]
        q, scale, full = outputs(6, 1031, torch.int8)
        qq = torch.zeros(6, 1100, dtype=torch.int8, device="cuda")[:, offset:offset + 1031]
        capi.rmsnorm_q8_run(x, weight, qq, scale, EPS, residual=residual, residual_out=out)
        h, y = norm64(x, weight, EPS, residual)
        check_codes(qq, scale, y, CODE_ERR, 2.0 ** -17)
        check_values(out, h, h.abs() * U)
        assert float(buf[:, :offset].abs().max()) == 0.0


@pytest.mark.parametrize("cols", [5, 255, 257, 4099, 12501, 25001, 32765])
@pytest.mark.parametrize("dtype", VALUE_TYPES)
def test_loose_rows(dtype, cols):
    """Rows of odd pitches, on every offset inside 16 bytes, narrow and too wide for two copies."""
    x = values(1, 9 * (cols + 3), dtype, 20)[0].view(9, cols + 3)[:, :cols]
    r = values(1, 9 * (cols + 1), dtype, 21)[0].view(9, cols + 1)[:, :cols]
    weight = values(1, cols + 1, dtype, 22)[0, 1:]
    for residual in (None, r):
        q, scale, out = run_norm(x, weight, torch.float8_e4m3fn, residual)
        h, y = norm64(x, weight, EPS, residual)
        check_codes(q, scale, y, CODE_ERR, 2.0 ** -17, f"{cols}")
        if residual is not None:
            check_values(out, h, h.abs() * U)
    q, scale, full = outputs(9, cols, torch.int8)
    flat = values(1, 18 * cols + 1, dtype, 23)[0, 1:]
    gate, up = flat[:9 * cols].view(9, cols), flat[9 * cols:].view(9, cols)
    capi.silu_mul_q8_run(gate, up, q, scale)
    check_guard(full, cols)
    err = 2 * (float(gate.abs().max()) + 4) * U + 16 * U
    check_codes(q, scale, act64(gate, up), 2 * err, err)


@pytest.mark.parametrize("cols", [6, 254, 258, 2050, 4098, 8194, 12502, 32766])
@pytest.mark.parametrize("dtype", VALUE_TYPES)
def test_pair_rows(dtype, cols):
    """Rows that start on pairs of elements, but not on 16 bytes."""
    x = values(1, 9 * (cols + 4), dtype, 30)[0].view(9, cols + 4)[:, 2:cols + 2]
    r = values(1, 9 * (cols + 2), dtype, 31)[0].view(9, cols + 2)[:, :cols]
    weight = values(1, cols + 2, dtype, 32)[0, 2:]
    for residual in (None, r):
        for code_dtype in CODE_TYPES:
            q, scale, out = run_norm(x, weight, code_dtype, residual)
            h, y = norm64(x, weight, EPS, residual)
            check_codes(q, scale, y, CODE_ERR, 2.0 ** -17, f"{cols}")
            if residual is not None:
                check_values(out, h, h.abs() * U)
    q, scale, full = outputs(9, cols, torch.int8)
    flat = values(1, 18 * cols + 2, dtype, 33)[0, 2:]
    gate, up = flat[:9 * cols].view(9, cols), flat[9 * cols:].view(9, cols)
    capi.silu_mul_q8_run(gate, up, q, scale)
    check_guard(full, cols)
    err = 2 * (float(gate.abs().max()) + 4) * U + 16 * U
    check_codes(q, scale, act64(gate, up), 2 * err, err)


@pytest.mark.parametrize("cols", [64, 1000, 1001, 4096, 8192])
def test_norm_in_place(cols):
    """residual_out may be the residual or x itself."""
    for dtype in VALUE_TYPES:
        x, r = values(37, cols, dtype, 1), values(37, cols, dtype, 2)
        weight = torch.ones(cols, dtype=dtype, device="cuda")
        q0, s0, out0 = run_norm(x, weight, torch.int8, r)
        for target in ("residual", "x"):
            xc, rc = x.clone(), r.clone()
            q, scale, _ = outputs(37, cols, torch.int8)
            into = rc if target == "residual" else xc
            capi.rmsnorm_q8_run(xc, weight, q, scale, EPS, residual=rc, residual_out=into)
            assert torch.equal(q, q0) and torch.equal(scale, s0) and torch.equal(into, out0)


def test_norm_zero_tiny_and_large_rows():
    cols = 1024
    x = values(8, cols, torch.float32, 3)
    x[0] = 0.0
    x[1] *= 1e-30
    x[2] *= 1e-42   # subnormal
    x[3] *= 1e15
    x[4] = 0.0
    x[4, 17] = -3.0
    weight = torch.ones(cols, device="cuda")
    for code_dtype in CODE_TYPES:
        q, scale, _ = run_norm(x, weight, code_dtype)
        assert float(scale[0]) == 1.0 and float(q[0].float().abs().max()) == 0.0
        y = norm64(x, weight, EPS)[1]
        keep = [3, 4, 5, 6, 7]
        check_codes(q[keep], scale[keep], y[keep], CODE_ERR, 2.0 ** -17)
        # rows whose values fall under eps: fp32 subnormals keep fewer bits
        # (row 1: values of about 1e-27; row 2's are subnormal themselves)
        check_codes(q[1:2], scale[1:2], y[1:2], CODE_ERR, 2.0 ** -17)
        assert bool(torch.isfinite(scale[2])) and float(q[2].float().abs().max()) > 0.0


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_rows_not_finite_stay_alone(bad):
    """A row with a NaN or an infinity: scale NaN, codes 0; every other row as without it."""
    for dtype in VALUE_TYPES:
        for code_dtype in CODE_TYPES:
            x, r = values(5, 777, dtype, 4), values(5, 777, dtype, 5)
            weight = torch.ones(777, dtype=dtype, device="cuda")
            q0, s0, _ = run_norm(x, weight, code_dtype, r)
            x[2, 776] = bad
            q, scale, out = run_norm(x, weight, code_dtype, r)
            keep = [0, 1, 3, 4]
            assert torch.equal(scale[keep], s0[keep])
            assert torch.equal(q[keep].view(torch.uint8), q0[keep].view(torch.uint8))
            assert bool(torch.isnan(scale[2])) and float(q[2].float().abs().max()) == 0.0
            assert not bool(torch.isfinite(out[2, 776]))
            up = values(5, 777, dtype, 6)
            qa, sa, _ = outputs(5, 777, code_dtype)
            capi.silu_mul_q8_run(r, up, qa, sa)
            up[3, 0] = bad
            qb, sb, _ = outputs(5, 777, code_dtype)
            capi.silu_mul_q8_run(r, up, qb, sb)
            keep = [0, 1, 2, 4]
            assert torch.equal(sa[keep], sb[keep])
            assert torch.equal(qa[keep].view(torch.uint8), qb[keep].view(torch.uint8))
            assert bool(torch.isnan(sb[3])) and float(qb[3].float().abs().max()) == 0.0


def test_norm_sum_of_squares_overflow_is_marked():
    x = torch.full((2, 64), 1e19, device="cuda")
    x[1] = 1.0
    q, scale, _ = run_norm(x, torch.ones(64, device="cuda"), torch.int8)
    assert bool(torch.isnan(scale[0])) and float(scale[1]) == pytest.approx(1 / 127, rel=1e-6)


@pytest.mark.parametrize("code_dtype", CODE_TYPES)
@pytest.mark.parametrize("dtype", VALUE_TYPES)
def test_act_sizes(dtype, code_dtype):
    for i, (rows, cols) in enumerate(SIZES):
        both = values(rows, 2 * cols, dtype, 400 + i, pitch_extra=i % 2, spread=3.0)
        gate, up = both[:, :cols], both[:, cols:]
        q, scale, full = outputs(rows, cols, code_dtype)
        capi.silu_mul_q8_run(gate, up, q, scale)
        check_guard(full, cols)
        err = 2 * (float(gate.abs().max()) + 4) * U + 16 * U
        check_codes(q, scale, act64(gate, up), 2 * err, err, f"{rows}x{cols}")


def test_act_far_arguments():
    """Gates far on either side: silu is 0 on the left, the identity on the right."""
    gate = torch.tensor([[-200.0, -100.0, -90.0, 0.0, 90.0, 200.0, 1e4, -1e4]], device="cuda")
    up = torch.ones_like(gate)
    q, scale, _ = outputs(1, 8, torch.int8)
    capi.silu_mul_q8_run(gate, up, q, scale)
    assert float(scale[0]) == pytest.approx(1e4 / 127, rel=1e-6)
    assert q[0].tolist() == [0, 0, 0, 0, 1, 3, 127, 0]


def test_rows_empty():
    x = torch.empty(0, 64, device="cuda")
    q = torch.empty(0, 64, dtype=torch.int8, device="cuda")
    capi.rmsnorm_q8_run(x, torch.ones(64, device="cuda"), q, torch.empty(0, device="cuda"), EPS)
    capi.silu_mul_q8_run(x, x, q, torch.empty(0, device="cuda"))
    torch.cuda.synchronize()


def test_rows_many():
    """More rows than blocks are resident at once, each with its own scale."""
    x = values(40001, 130, torch.bfloat16, 8)
    x *= torch.rand(40001, 1, device="cuda") + 0.5
    weight = torch.ones(130, device="cuda")
    q, scale, _ = run_norm(x, weight, torch.int8)
    check_codes(q, scale, norm64(x, weight, EPS)[1], CODE_ERR, 2.0 ** -17)


def test_rows_offsets_past_32_bits():
    """Rows whose byte and element offsets pass 2^31 and 2^32."""
    pitch = 700_000_000
    buf = torch.empty(4 * pitch, dtype=torch.bfloat16, device="cuda")
    x = buf.view(4, pitch)[:, :256]
    x.copy_(values(4, 256, torch.bfloat16, 11))
    weight = torch.ones(256, device="cuda")
    q, scale, _ = run_norm(x, weight, torch.int8)
    check_codes(q, scale, norm64(x, weight, EPS)[1], CODE_ERR, 2.0 ** -17)


def test_rows_on_a_side_stream_and_in_a_graph():
    x, r = values(64, 4096, torch.bfloat16, 12), values(64, 4096, torch.bfloat16, 13)
    weight = torch.ones(4096, dtype=torch.bfloat16, device="cuda")
    q0, s0, out0 = run_norm(x, weight, torch.float8_e4m3fn, r)
    s = torch.cuda.Stream()
    xs = torch.zeros_like(x)
    q, scale, _ = outputs(64, 4096, torch.float8_e4m3fn)
    out = torch.empty_like(x)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        xs.copy_(x)
        capi.rmsnorm_q8_run(xs, weight, q, scale, EPS, residual=r, residual_out=out)
    torch.cuda.synchronize()
    assert torch.equal(q.view(torch.uint8), q0.view(torch.uint8)) and torch.equal(out, out0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        capi.rmsnorm_q8_run(xs, weight, q, scale, EPS, residual=r, residual_out=out)
    xs.mul_(2.0)
    r2 = r.clone()
    r.mul_(2.0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, 2 * out0)
    # doubled values: the same codes but for eps, a scale of the same size
    assert float((scale / s0 - 1).abs().max()) < 1e-3
    r.copy_(r2)


def test_refusals():
    x = torch.zeros(4, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    q = torch.zeros(4, 64, dtype=torch.int8, device="cuda")
    s = torch.zeros(4, device="cuda")
    for call in (
            lambda: capi.rmsnorm_q8_run(x, w[:63], q, s, EPS),
            lambda: capi.rmsnorm_q8_run(x, w, q[:, :63], s, EPS),
            lambda: capi.rmsnorm_q8_run(x, w, q, s[:3], EPS),
            lambda: capi.rmsnorm_q8_run(x, w, q.to(torch.int16), s, EPS),
            lambda: capi.rmsnorm_q8_run(x.double(), w, q, s, EPS),
            lambda: capi.rmsnorm_q8_run(x.t(), w[:4], q.t(), torch.zeros(64, device="cuda"), EPS),
            lambda: capi.rmsnorm_q8_run(x.cpu(), w, q, s, EPS),
            lambda: capi.rmsnorm_q8_run(x, w, q, s.double(), EPS),
            lambda: capi.rmsnorm_q8_run(x, w, q, s, EPS, residual=x.half(), residual_out=x),
            lambda: capi.silu_mul_q8_run(x, x[:, :63], q, s),
            lambda: capi.silu_mul_q8_run(x, x.half(), q, s),
            lambda: capi.silu_mul_q8_run(x, x, q, s.half())):
        with pytest.raises(ValueError):
            call()
    for call, status in (
            (lambda: capi.rmsnorm_q8_run(x, w, q, s, EPS, residual=x), capi.CONV3D_EINVAL),
            (lambda: capi.rmsnorm_q8_run(x, w, q, s, EPS, residual_out=x), capi.CONV3D_EINVAL),
            (lambda: capi.rmsnorm_q8_run(x, w, q, s, -1.0), capi.CONV3D_EINVAL),
            (lambda: capi.rmsnorm_q8_run(x, w, q, s, float("nan")), capi.CONV3D_EINVAL),
            (lambda: capi.rmsnorm_q8_run(torch.zeros(1, 32769, device="cuda"),
                                         torch.zeros(32769, device="cuda"),
                                         torch.zeros(1, 32769, dtype=torch.int8, device="cuda"),
                                         s[:1], EPS), capi.CONV3D_EUNSUPPORTED)):
        with pytest.raises(capi.Conv3dFp8Error) as e:
            call()
        assert e.value.status == status
