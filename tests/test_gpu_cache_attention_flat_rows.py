"""Rows of equal values in a cache: zeros, or any constant in 4 bits, which are stored with codes of 0 and the scale 1,
whatever the size of the rows beside them."""
import pytest
import torch

from fp8_implicit_gemm_gb300 import capi, q8
from _attention_common import CODE_ARG, CODES, attention64, check_attention, codes64, fill_cache, randn, values64

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16]
WEIGHT_ROUND = 2.0 ** -11


def put(cache, codes, name, place, row):
    """Rows [n, kv_heads, dim] at places of a cache whose pages lie in order."""
    q, scale, lowest = codes64(row, codes)
    page, at = place // cache.page_size, place % cache.page_size
    as_bytes = getattr(cache, name + "_codes").view(torch.uint8)
    if codes == "i4":
        b = q.to(torch.uint8)
        as_bytes[page, :, at] = b[..., 0::2] | (b[..., 1::2] << 4)
        scale = torch.stack([scale, lowest], dim=-1)
    else:
        as_bytes[page, :, at] = q.to(cache.k_codes.dtype).view(torch.uint8)
    getattr(cache, name + "_scale")[page, :, at] = scale.float()


def verify(cache, codes, q, n, tokens=1, scale=None, page=16):
    heads, dim = q.shape[1:]
    table = torch.arange(cache.pages, dtype=torch.int32, device="cuda")[None]
    attend = q8.CacheAttention(cache, heads, max_tokens=tokens, scale=scale)
    o = attend(q, table, torch.tensor([n], dtype=torch.int32, device="cuda"), torch.full_like(q, 7.0))
    assert attend.check() == capi.CONV3D_OK
    k, v = [values64(cache, name, codes).transpose(1, 2).flatten(0, 1)[:n] for name in "kv"]
    limits = (n - tokens + 1 + torch.arange(tokens, device="cuda")).clamp(min=0)
    want, size, worst = attention64(q, k, v, limits, dim ** -0.5 if scale is None else scale)
    check_attention(o, want, size, worst, WEIGHT_ROUND, n)
    return o


def cache_of(codes, n, kv, dim, spread=1.0, page=16, seed=1):
    cache = q8.CacheQ8.empty(-(-n // page), page, kv, dim, CODE_ARG[codes])
    fill_cache(cache, codes, seed)
    if spread != 1.0:
        cache.v_scale.mul_(spread)
    return cache


@pytest.mark.parametrize("codes", CODES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,place", [(40, 3), (4096, 0), (4096, 4095), (32768, 1000)])
@pytest.mark.parametrize("nats", [3.0, 13.0, 40.0, 300.0])
def test_a_row_of_zeros_that_takes_the_weight(codes, dtype, n, place, nats):
    """A key whose score is so far above all others, its value zeros (a sink): the others' values keep their share. Their
    scales are about 0.004 or 0.15, the zeros' is 1."""
    dim, kv = 64, 2
    cache = cache_of(codes, n, kv, dim, 0.5)
    cache.k_scale.mul_(2.0 ** -6)
    q = torch.full((1, 8, dim), 1.0, device="cuda").to(dtype) + randn(1, 8, dim, dtype=dtype, seed=5) / 16
    at = torch.tensor([place], device="cuda")
    put(cache, codes, "k", at, torch.full((1, kv, dim), nats / 8.0, device="cuda") * (1 + 0.01 * randn(1, kv, dim, seed=6)))
    put(cache, codes, "v", at, torch.zeros(1, kv, dim, device="cuda"))
    verify(cache, codes, q, n)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("value", [1e-8, 1e-6, 2.4e-7, 1e-3, -1e-5, 0.3, 1e4, 0.0])
@pytest.mark.parametrize("n", [1, 2, 100])
def test_constant_rows_of_4_bits(dtype, value, n):
    """All values of a row alike, all rows or one: what is read back is that value, and so is what attention gives."""
    dim = 128
    cache = cache_of("i4", n, 1, dim)
    places = torch.arange(n, device="cuda")
    put(cache, "i4", "v", places, torch.full((n, 1, dim), value, device="cuda"))
    q = randn(1, 4, dim, dtype=dtype, seed=5)
    o = verify(cache, "i4", q, n)
    stored = torch.tensor(value, dtype=torch.float32)
    # sums and quotients of n equal values in fp32 err by (n / 4 + 8) * 2^-23 of them, then the output is rounded
    info = torch.finfo(dtype)
    bound = abs(float(stored)) * ((n / 4 + 8) * 2.0 ** -23 + info.eps / 2) * 1.001 + info.smallest_normal * info.eps / 2
    assert float((o.double() - float(stored)).abs().max()) <= bound


@pytest.mark.parametrize("codes", CODES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("size", [1e-5, 1e-8, 1.0, 1e5])
@pytest.mark.parametrize("tokens,heads", [(1, 4), (3, 12)])
def test_rows_of_zeros_among_others(codes, dtype, size, tokens, heads):
    """A third of the rows of v is zeros (in 4 bits: another third constant), beside rows of any size."""
    n, dim, kv = 1000, 128, 2
    cache = cache_of(codes, n, kv, dim, size if dtype == torch.bfloat16 else min(size, 1.0))
    size = size if dtype == torch.bfloat16 else min(size, 1.0)
    g = torch.Generator(device="cuda").manual_seed(3)
    order = torch.randperm(n, generator=g, device="cuda")
    put(cache, codes, "v", order[:333], torch.zeros(333, kv, dim, device="cuda"))
    if codes == "i4":
        put(cache, codes, "v", order[333:600], (size * randn(267, kv, 1, seed=7)).expand(-1, -1, dim))
    verify(cache, codes, randn(tokens, heads, dim, dtype=dtype, seed=5), n, tokens)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim,heads", [(64, 2), (128, 12), (256, 1)])
@pytest.mark.parametrize("value", [0.0, 0.7, -0.1])
@pytest.mark.parametrize("size,n", [(1e-3, 200), (1e-4, 200), (1e-4, 2), (1.0, 50)])
def test_constant_keys_of_4_bits(dtype, dim, heads, value, size, n):
    """Small keys beside large queries: a constant key's score is its value times the sum of q, nothing of its scale of 1."""
    cache = cache_of("i4", n, 1, dim)
    cache.k_scale.mul_(size)
    places = torch.arange(0, n, 2, device="cuda")
    put(cache, "i4", "k", places, torch.full((places.numel(), 1, dim), value * size, device="cuda"))
    verify(cache, "i4", (randn(1, heads, dim, seed=5) / size).to(dtype), n)


@pytest.mark.parametrize("codes", CODES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shift", [0.0, 30.0, -30.0])
def test_scales_of_1_beside_codes(codes, dtype, shift):
    """Rows whose scale is 1 and whose codes are not all 0, one code of them or all, are ordinary rows."""
    n, dim = 300, 64
    cache = cache_of(codes, n, 1, dim)
    for t in (cache.k_scale, cache.v_scale):
        t.view(t.shape[:3] + (-1,))[..., 0] = 1.0
    as_bytes = cache.v_codes.view(torch.uint8)
    as_bytes[::2] = 0
    as_bytes[::2, :, :, 5] = 0x30  # one code of the row
    cache.k_scale.mul_(2.0 ** -5)
    if codes == "i4":
        cache.k_scale[::3, ..., 0] = 1.0
    q = randn(1, 4, dim, dtype=dtype, seed=5)
    q[..., 0] += shift
    verify(cache, codes, q, n)
    cache.v_codes.view(torch.uint8).zero_()  # and nothing but rows of zeros
    verify(cache, codes, q, n)


@pytest.mark.parametrize("codes", CODES)
@pytest.mark.parametrize("dtype", TYPES)
def test_rows_do_not_depend_on_their_neighbours(codes, dtype):
    """A head's output is the same bit by bit beside heads whose scores are larger, with rows of zeros in the cache."""
    n, dim = 500, 128
    cache = cache_of(codes, n, 1, dim, 0.1)
    put(cache, codes, "v", torch.arange(0, n, 3, device="cuda"), torch.zeros(167, 1, dim, device="cuda"))
    table = torch.arange(cache.pages, dtype=torch.int32, device="cuda")[None]
    length = torch.tensor([n], dtype=torch.int32, device="cuda")
    attend = q8.CacheAttention(cache, 8)
    q = randn(1, 8, dim, dtype=dtype, seed=5)
    want = attend(q, table, length, torch.empty_like(q)).clone()
    for other in range(1, 8):
        p = q.clone()
        p[:, other:] *= 7
        assert torch.equal(attend(p, table, length, torch.empty_like(q))[:, :other], want[:, :other])


@pytest.mark.parametrize("codes", CODES)
def test_rows_of_zeros_as_the_library_writes_them(codes):
    """The same rows through heads_q8_run: what it leaves for rows of equal values is what attention takes as such."""
    n, dim, kv = 100, 128, 2
    k, v = randn(n, kv, dim, dtype=torch.bfloat16, seed=1), randn(n, kv, dim, dtype=torch.bfloat16, seed=2) / 256
    v[::2] = 0
    v[1] = 2.0 ** -20
    k[7] = 0
    cache = q8.CacheQ8.empty(7, 16, kv, dim, CODE_ARG[codes])
    capi.heads_q8_run(k=k, v=v, cache=cache, slots=torch.arange(n, device="cuda"))
    verify(cache, codes, randn(1, 8, dim, dtype=torch.bfloat16, seed=5), n)
