"""Products of 8-bit codes with a scale for each token and channel, against 64-bit forms."""
import pytest
import torch

from fp8_implicit_gemm_gb300 import capi, q8
from _q8_common import CODE_TYPES, VALUE_TYPES, check_values, linear64, linear_err, padded

pytestmark = pytest.mark.gpu


def codes(rows, cols, dtype, seed, extra=0):
    """Codes over the whole range of the type (e4m3 without its NaNs), in padded rows whose padding
    holds codes that must not count (e4m3: NaN)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = padded(rows, cols, dtype, extra)
    full = out.as_strided((rows, out.stride(0)), (out.stride(0), 1))
    full.view(torch.uint8).fill_(0x7F)
    if dtype == torch.int8:
        out.copy_(torch.randint(-128, 128, (rows, cols), generator=g, device="cuda"))
    else:
        v = torch.randn(rows, cols, generator=g, device="cuda") * 100
        out.copy_(v.clamp(-448, 448))
    return out


def scales(n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand(n, generator=g, device="cuda") * 0.02 + 1e-3


def case(M, N, K, code_dtype, y_dtype, seed, bias_dtype=None, extra=0):
    x, w = codes(M, K, code_dtype, seed, extra), codes(N, K, code_dtype, seed + 1, extra)
    sx, sw = scales(M, seed + 2), scales(N, seed + 3)
    bias = None
    if bias_dtype is not None:
        bias = (torch.randn(N, generator=torch.Generator(device="cuda").manual_seed(seed + 4),
                            device="cuda") * 10).to(bias_dtype)
    return x, sx, w, sw, bias


def run(x, sx, w, sw, bias, y_dtype, max_rows=None, y_extra=5, **options):
    M, N = x.shape[0], w.shape[0]
    full = torch.full((M + 2, N + y_extra), float("nan"), dtype=y_dtype, device="cuda")
    y = full[1:M + 1, :N]
    plan = capi.linear_q8_plan(max_rows or M, N, w.shape[1], capi.q8_code_type(w.dtype), 0,
                               **options)
    try:
        capi.linear_q8_run(plan, x, sx, w, sw, y, bias)
        assert capi.linear_q8_check(plan) == capi.CONV3D_OK
        again = torch.empty_like(y)
        for _ in range(2):
            capi.linear_q8_run(plan, x, sx, w, sw, again, bias)
        assert capi.linear_q8_check(plan) == capi.CONV3D_OK
    finally:
        capi.linear_q8_destroy(plan)
    assert bool(torch.isnan(full[0]).all()) and bool(torch.isnan(full[M + 1]).all())
    assert bool(torch.isnan(full[:, N:]).all())
    assert same_bits(y, again), "two runs differ"
    return y


def same_bits(a, b):
    as_int = torch.int32 if a.dtype == torch.float32 else torch.int16
    return torch.equal(a.contiguous().view(as_int), b.contiguous().view(as_int))


def check(M, N, K, code_dtype, y_dtype, seed, bias_dtype=None, extra=0, max_rows=None,
          y_extra=5, **options):
    x, sx, w, sw, bias = case(M, N, K, code_dtype, y_dtype, seed, bias_dtype, extra)
    y = run(x, sx, w, sw, bias, y_dtype, max_rows, y_extra, **options)
    want, mag = linear64(x, sx, w, sw, bias)
    check_values(y, want, linear_err(mag, K, code_dtype), f"{M}x{N}x{K} {options}")


# one token, a few, many; widths and lengths around every tile and vector size
SIZES = [(1, 1, 1), (1, 5, 7), (1, 16, 16), (1, 33, 64), (1, 4096, 1024), (2, 300, 1000),
         (3, 17, 129), (7, 256, 512), (8, 128, 4096), (9, 1000, 96), (15, 64, 63), (16, 500, 2048),
         (17, 129, 65), (31, 257, 1024), (32, 512, 256), (33, 100, 1001), (48, 640, 384),
         (64, 1024, 4096), (65, 130, 127), (100, 260, 100), (127, 255, 128), (128, 256, 1024),
         (129, 511, 130), (200, 1000, 200), (255, 384, 2049), (257, 513, 1025), (300, 2500, 1001),
         (512, 768, 640), (1000, 300, 5000), (2049, 1100, 300)]


@pytest.mark.parametrize("code_dtype", CODE_TYPES)
@pytest.mark.parametrize("y_dtype", VALUE_TYPES)
def test_sizes(code_dtype, y_dtype):
    for i, (M, N, K) in enumerate(SIZES):
        check(M, N, K, code_dtype, y_dtype, 1000 + 10 * i,
              [None, torch.float32, torch.bfloat16, torch.float16][i % 4], extra=i % 3,
              max_rows=M + (i % 2) * 777)


@pytest.mark.parametrize("code_dtype", CODE_TYPES)
@pytest.mark.parametrize("M", [1, 4, 24, 96, 700])
def test_every_short_length(code_dtype, M):
    """K from 1 past the first tiles: the last step of every length is cut where it should be."""
    for K in list(range(1, 36)) + [47, 48, 49, 63, 64, 65, 79, 80, 81, 127, 128, 129, 191, 192, 193]:
        check(M, 72, K, code_dtype, torch.float32, 7 * K)


@pytest.mark.parametrize("code_dtype", CODE_TYPES)
def test_large(code_dtype):
    check(4096, 4096, 1024, code_dtype, torch.float32, 77)
    check(1111, 8200, 4100, code_dtype, torch.bfloat16, 78, torch.float32)


@pytest.mark.parametrize("code_dtype", CODE_TYPES)
@pytest.mark.parametrize("block_t", [32, 64, 96, 128, 160, 192, 224, 256])
def test_every_tile(code_dtype, block_t):
    """Every tile, whole and in slices, on one pair of CTAs and on many, with stores of one channel
    and of four, and with fewer tokens than a tile."""
    if code_dtype == torch.int8 and block_t > 192:
        pytest.skip("int8 tiles have up to 192 tokens")
    for M in (block_t - 31, block_t, 3 * block_t - 5):
        for i, (N, K) in enumerate([(300, 1000), (520, 1536), (256, 130)]):
            check(M, N, K, code_dtype, VALUE_TYPES[i], 31 * M + i, torch.float32, kernel=2,
                  block_t=block_t, splits=1, y_extra=4 * (i % 2))
            check(M, N, K, code_dtype, VALUE_TYPES[i], 31 * M + i, kernel=2, block_t=block_t,
                  splits=1, max_ctas=2)
            for splits in (2, 3, 4):
                if -(-K // 256) >= splits:
                    check(M, N, K, code_dtype, VALUE_TYPES[i], 31 * M + i, torch.float32, kernel=2,
                          block_t=block_t, splits=splits, y_extra=4 * (i % 2))


@pytest.mark.parametrize("code_dtype", CODE_TYPES)
def test_few_tokens_on_both_kernels(code_dtype):
    for M in (1, 5, 8, 9, 16):
        for kernel in (1, 2):
            check(M, 777, 1030, code_dtype, torch.float32, 13 * M, kernel=kernel)


@pytest.mark.parametrize("code_dtype", CODE_TYPES)
def test_a_wait_that_runs_out_is_reported(code_dtype):
    """The loader's first copy left out (a test flag): every wait on it runs out of its 50 ms, the
    kernel ends, the check reports it once, and the plan's next user is not affected."""
    x, sx, w, sw, _ = case(100, 300, 1000, code_dtype, torch.float32, 90)
    for splits in (1, 2):
        plan = capi.linear_q8_plan(100, 300, 1000, capi.q8_code_type(code_dtype), 0, block_t=64,
                                   splits=splits, wait_timeout_ms=50, debug_flags=1)
        y = torch.zeros(100, 300, device="cuda")
        capi.linear_q8_run(plan, x, sx, w, sw, y)
        assert capi.linear_q8_check(plan) == capi.CONV3D_EDEVICE
        assert capi.linear_q8_check(plan) == capi.CONV3D_OK
        capi.linear_q8_destroy(plan)
    check(100, 300, 1000, code_dtype, torch.float32, 90)


def test_options_that_leave_no_tiling():
    x, sx, w, sw, _ = case(40, 64, 200, torch.int8, torch.float32, 91)
    y = torch.zeros(40, 64, device="cuda")
    for options in (dict(block_t=96), dict(splits=4)):
        plan = capi.linear_q8_plan(40, 64, 200, capi.Q8_INT8, 0, **options)
        with pytest.raises(capi.Conv3dFp8Error) as e:
            capi.linear_q8_run(plan, x, sx, w, sw, y)
        assert e.value.status == capi.CONV3D_EUNSUPPORTED
        capi.linear_q8_destroy(plan)
    for options in (dict(block_t=33), dict(block_t=288), dict(splits=5), dict(kernel=3),
                    dict(max_ctas=-1), dict(wait_timeout_ms=-1)):
        with pytest.raises(capi.Conv3dFp8Error) as e:
            capi.linear_q8_plan(40, 64, 200, capi.Q8_INT8, 0, **options)
        assert e.value.status == capi.CONV3D_EINVAL
    with pytest.raises(capi.Conv3dFp8Error) as e:
        capi.linear_q8_plan(40, 64, 200, capi.Q8_INT8, 0, kernel=1)
    assert e.value.status == capi.CONV3D_EUNSUPPORTED


def test_int8_extremes_are_exact():
    """Sums at the edge of what 32 bits of a float hold exactly: 1024 products of -128 * -128."""
    for M in (1, 20, 300):
        x = torch.full((M, 1024), -128, dtype=torch.int8, device="cuda")
        w = torch.full((136, 1024), -128, dtype=torch.int8, device="cuda")
        w[5] = 127
        one = torch.ones(M, device="cuda"), torch.ones(136, device="cuda")
        y = run(x, one[0], w, one[1], None, torch.float32)
        want = (x[:1].double() @ w.double().t())[0]
        assert bool((y.double() == want).all())


def test_int8_long_sums():
    """A sum of 2^28: each instruction may cut 2^-23 of it."""
    for M in (1, 40, 256):
        x = torch.full((M, 16384), 127, dtype=torch.int8, device="cuda")
        w = torch.full((64, 16384), 127, dtype=torch.int8, device="cuda")
        y = run(x, torch.ones(M, device="cuda"), w, torch.ones(64, device="cuda"), None,
                torch.float32)
        want = 127.0 * 127.0 * 16384
        assert float((y.double() - want).abs().max()) <= (16384 / 16) * 2.0 ** -23 * want


@pytest.mark.parametrize("M", [1, 12, 40, 300])
def test_not_finite_stays_in_its_row_and_column(M):
    x, sx, w, sw, _ = case(M, 200, 300, torch.int8, torch.float32, 5)
    y0 = run(x, sx, w, sw, None, torch.float32)
    sx[M // 2] = float("nan")
    sw[33] = float("inf")
    y = run(x, sx, w, sw, None, torch.float32)
    assert bool(torch.isnan(y[M // 2]).all())
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[M // 2] = False
    keep[:, 33] = False
    assert torch.equal(y[keep], y0[keep])
    assert not bool(torch.isfinite(y[:, 33]).any())


@pytest.mark.parametrize("M", [1, 12, 40, 300])
def test_e4m3_nan_codes(M):
    """A NaN code makes its row (of x) or column (of w) NaN and no other element."""
    x, sx, w, sw, _ = case(M, 200, 300, torch.float8_e4m3fn, torch.float32, 6)
    y0 = run(x, sx, w, sw, None, torch.float32)
    x.view(torch.uint8)[M // 2, 299] = 0x7F
    w.view(torch.uint8)[199, 0] = 0xFF
    y = run(x, sx, w, sw, None, torch.float32)
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[M // 2] = False
    keep[:, 199] = False
    assert bool(torch.isnan(y[~keep]).all())
    assert torch.equal(y[keep], y0[keep])


def test_one_row_of_any_pitch_and_rows_of_a_larger_matrix():
    w, sw = codes(96, 80, torch.int8, 1), scales(96, 2)
    big = codes(64, 160, torch.int8, 3)
    sx = scales(64, 4)
    x = big[::4, 16:96]   # every fourth row, from a column inside
    y = run(x, sx[:16].contiguous(), w, sw, None, torch.float32)
    want, mag = linear64(x, sx[:16], w, sw)
    check_values(y, want, linear_err(mag, 80, torch.int8))
    one = torch.as_strided(big, (1, 80), (3, 1))
    y = run(one, sx[:1], w, sw, None, torch.float32)
    want, mag = linear64(one, sx[:1], w, sw)
    check_values(y, want, linear_err(mag, 80, torch.int8))


def test_fewer_rows_than_planned_and_none():
    x, sx, w, sw, _ = case(300, 512, 256, torch.int8, torch.float32, 8)
    plan = capi.linear_q8_plan(300, 512, 256, capi.Q8_INT8, 0)
    want, mag = linear64(x, sx, w, sw)
    try:
        for rows in (300, 1, 17, 0, 130, 64, 2, 299):
            y = torch.full((rows, 512), float("nan"), device="cuda")
            capi.linear_q8_run(plan, x[:rows], sx[:rows], w, sw, y)
            assert capi.linear_q8_check(plan) == capi.CONV3D_OK
            if rows:
                check_values(y, want[:rows], linear_err(mag[:rows], 256, torch.int8))
    finally:
        capi.linear_q8_destroy(plan)


@pytest.mark.parametrize("M", [1, 16, 64, 500])
@pytest.mark.parametrize("code_dtype", CODE_TYPES)
def test_plans_on_streams_of_their_own(M, code_dtype):
    """Three plans, three streams, many runs in flight: the same bits as one after the other."""
    sets = [case(M, 1000, 2000, code_dtype, torch.float32, 40 + k) for k in range(3)]
    want = [run(*s, torch.bfloat16) for s in sets]
    plans = [capi.linear_q8_plan(M, 1000, 2000, capi.q8_code_type(code_dtype), 0) for _ in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    ys = [[torch.empty(M, 1000, dtype=torch.bfloat16, device="cuda") for _ in range(8)]
          for _ in sets]
    torch.cuda.synchronize()
    for r in range(8):
        for s, p, st, y in zip(sets, plans, streams, ys):
            capi.linear_q8_run(p, s[0], s[1], s[2], s[3], y[r], None, st)
    torch.cuda.synchronize()
    for p, y, ref in zip(plans, ys, want):
        assert capi.linear_q8_check(p) == capi.CONV3D_OK
        capi.linear_q8_destroy(p)
        for v in y:
            assert torch.equal(v, ref)


@pytest.mark.parametrize("M", [1, 40, 500])
def test_graph(M):
    x, sx, w, sw, _ = case(M, 640, 1024, torch.int8, torch.float32, 60)
    ref = run(x, sx, w, sw, None, torch.float32)
    layer = q8.LinearQ8(w, sw, max_rows=M)
    y = torch.empty(M, 640, device="cuda")
    layer(x, sx, y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer(x, sx, y)
    y.fill_(float("nan"))
    sx.mul_(2.0)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert layer.check() == capi.CONV3D_OK
    assert torch.equal(y, 2 * ref)
    layer.close()


def test_offsets_past_32_bits():
    """Rows of x and y whose offsets pass 2^31 elements."""
    pitch = 800_000_000
    buf = torch.empty(4 * pitch, dtype=torch.int8, device="cuda")
    src, sx, w, sw, _ = case(4, 48, 256, torch.int8, torch.float32, 61)
    x = buf.view(4, pitch)[:, :256]
    x.copy_(src)
    y = torch.empty(4 * pitch, dtype=torch.bfloat16, device="cuda").view(4, pitch)[:, :48]
    plan = capi.linear_q8_plan(4, 48, 256, capi.Q8_INT8, 0)
    capi.linear_q8_run(plan, x, sx, w, sw, y)
    assert capi.linear_q8_check(plan) == capi.CONV3D_OK
    capi.linear_q8_destroy(plan)
    want, mag = linear64(src, sx, w, sw)
    check_values(y, want, linear_err(mag, 256, torch.int8))


def test_layer_lays_out_its_weights():
    """A weight whose rows are not laid out as the kernels read them is copied once."""
    x, sx, w, sw, _ = case(30, 50, 77, torch.int8, torch.float32, 62)
    layer = q8.LinearQ8(w.contiguous(), sw, max_rows=30)
    assert w.contiguous().stride(0) % 16 and layer.w.stride(0) % 16 == 0
    y = layer(x, sx, torch.empty(30, 50, device="cuda"))
    assert torch.equal(y, run(x, sx, w, sw, None, torch.float32))
    layer.close()
    layer.close()


@pytest.mark.parametrize("rows", [1, 3, 64, 333])
@pytest.mark.parametrize("code_dtype", CODE_TYPES)
def test_mlp_block(rows, code_dtype):
    """The three operators together, against fp64 on the same codes' weights. The block's own codes
    (one per value, of 7 or 3 bits) set its distance: within 4% (8 bits), 12% (e4m3) of the values'
    size, twice what independent rounding errors of two quantised products add up to."""
    torch.manual_seed(rows)
    dim, inner = 512, 1200
    w_gu = torch.randn(2 * inner, dim, device="cuda") / dim ** 0.5
    w_down = torch.randn(dim, inner, device="cuda") / inner ** 0.5
    weight = (1 + 0.1 * torch.randn(dim, device="cuda")).bfloat16()
    mlp = q8.MlpQ8(weight, w_gu, w_down, max_rows=400, codes=code_dtype)
    x, r = (torch.randn(rows, dim, device="cuda").bfloat16() for _ in range(2))
    residual = r.clone()
    y = mlp(x, residual, torch.empty_like(x))
    assert mlp.check() == capi.CONV3D_OK
    h = x.double() + r.double()
    assert torch.equal(residual, (x.float() + r.float()).bfloat16())
    a = h / torch.sqrt(h.square().mean(dim=1, keepdim=True) + 1e-6) * weight.double()
    g, u = (a @ w_gu.double().t()).chunk(2, dim=1)
    want = (torch.sigmoid(g) * g * u) @ w_down.double().t()
    err = float((y.double() - want).norm() / want.norm())
    assert err <= (0.04 if code_dtype == torch.int8 else 0.12), err
    with pytest.raises(ValueError):
        mlp(torch.zeros(401, dim, device="cuda"), residual, y)
    mlp.close()


def test_refusals():
    x, sx, w, sw, _ = case(8, 64, 64, torch.int8, torch.float32, 63)
    y = torch.zeros(8, 64, device="cuda")
    for args in ((0, 64, 64, 1, 0), (8, 0, 64, 1, 0), (8, 64, 0, 1, 0), (8, 64, 64, 0, 0),
                 (8, 64, 64, 3, 0), (8, 64, 64, 1, 5)):
        with pytest.raises(capi.Conv3dFp8Error) as e:
            capi.linear_q8_plan(*args)
        assert e.value.status == capi.CONV3D_EINVAL
    plan = capi.linear_q8_plan(8, 64, 64, capi.Q8_INT8, 0)

    def refused(error, *args, **kw):
        with pytest.raises(error) as e:
            capi.linear_q8_run(*args, **kw)
        if error is capi.Conv3dFp8Error:
            assert e.value.status == capi.CONV3D_EINVAL

    try:
        refused(ValueError, plan, x, sx, w.float(), sw, y)
        refused(ValueError, plan, x, sx, w.view(torch.uint8), sw, y)
        refused(ValueError, plan, x, sx[:7], w, sw, y)
        refused(ValueError, plan, x, sx, w, sw[:63], y)
        refused(ValueError, plan, x, sx, w, sw, y[:, :63])
        refused(ValueError, plan, x, sx, w, sw, y.double())
        refused(ValueError, plan, x.t().contiguous().t(), sx, w, sw, y)
        refused(ValueError, plan, x, sx, w, sw, y, bias=sw[:5])
        refused(ValueError, plan, x, sx.cpu(), w, sw, y)
        refused(ValueError, plan, x[:, :63], sx, w, sw, y)         # w has another length
        refused(capi.Conv3dFp8Error, plan, x[:, :32], sx, w[:, :32], sw, y)  # not the plan's
        refused(capi.Conv3dFp8Error, plan, x, sx, w[:32], sw[:32], y[:, :32])
        big = torch.zeros(9, 64, dtype=torch.int8, device="cuda")
        refused(capi.Conv3dFp8Error, plan, big, scales(9, 1), w, sw, torch.zeros(9, 64, device="cuda"))
        off = torch.zeros(8 * 72 + 16, dtype=torch.int8, device="cuda")
        refused(capi.Conv3dFp8Error, plan, off[:8 * 72].view(8, 72)[:, :64], sx, w, sw, y)
        refused(capi.Conv3dFp8Error, plan, off[8:8 + 512].view(8, 64), sx, w, sw, y)
        refused(capi.Conv3dFp8Error, 0, x, sx, w, sw, y)
        e4 = codes(8, 64, torch.float8_e4m3fn, 1), codes(64, 64, torch.float8_e4m3fn, 1)
        refused(capi.Conv3dFp8Error, plan, e4[0], sx, e4[1], sw, y)  # a plan for int8 codes
    finally:
        capi.linear_q8_destroy(plan)


# every way the kernel for few tokens divides the channels, the warps and the tokens
@pytest.mark.parametrize("code_dtype", CODE_TYPES)
@pytest.mark.parametrize("M,N,K", [(3, 100, 200), (1, 2432, 1024), (3, 70, 1300), (5, 2500, 300),
                                   (7, 4864, 2050), (8, 4900, 2100), (5, 9731, 130), (2, 9731, 600),
                                   (12, 80, 8300), (9, 2500, 200), (16, 4900, 200), (13, 9731, 200)])
def test_few_tokens_of_every_shape(code_dtype, M, N, K):
    check(M, N, K, code_dtype, torch.bfloat16, seed=M + N, bias_dtype=torch.float32, kernel=1)


@pytest.mark.parametrize("M,N,K", [(17, 100, 300), (24, 4864, 150), (21, 4900, 1200), (25, 100, 300),
                                   (32, 2432, 150), (29, 2500, 1200), (27, 9731, 60)])
def test_few_tokens_of_every_shape_int8(M, N, K):
    check(M, N, K, torch.int8, torch.float16, seed=M + N, kernel=1)


# y's rows anywhere on the 16-byte grid, whole tiles and ragged ones of channels and tokens
@pytest.mark.parametrize("y_dtype", VALUE_TYPES)
@pytest.mark.parametrize("y_extra", range(8))
def test_any_alignment_of_y(y_dtype, y_extra):
    for M, N in ((40, 256), (77, 300), (33, 129), (130, 511)):
        check(M, N, 150, torch.int8, y_dtype, seed=M, y_extra=y_extra, kernel=2, splits=1)
        check(M, N, 150, torch.float8_e4m3fn, y_dtype, seed=M, y_extra=y_extra, kernel=2, splits=1)


def test_layer_holds_its_weights():
    """A layer reads the memory it was made with, whatever becomes of the caller's tensors."""
    x, sx, w, sw, bias = case(20, 300, 256, torch.int8, torch.float32, 90, torch.float32)
    want, mag = linear64(x, sx, w, sw, bias)
    w = w.clone(memory_format=torch.contiguous_format)
    layer = q8.LinearQ8(w, sw, bias=bias, max_rows=20)
    w.data = torch.zeros(1, 1, dtype=torch.int8, device="cuda")
    sw.data = torch.zeros(1, device="cuda")
    del bias
    fill = [torch.full((300, 256), 55, dtype=torch.int8, device="cuda") for _ in range(4)]
    y = layer(x, sx, torch.empty(20, 300, device="cuda"))
    assert layer.check() == capi.CONV3D_OK and len(fill) == 4
    check_values(y, want, linear_err(mag, 256, torch.int8), "held")
    with pytest.raises(ValueError):
        layer(x[:, :255], sx, y)
    with pytest.raises(ValueError):
        layer(x.view(torch.float8_e4m3fn), sx, y)
    with pytest.raises(ValueError):
        layer(x, sx, y[:, :299])
    layer.close()
