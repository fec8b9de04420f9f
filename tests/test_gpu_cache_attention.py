"""Attention of the newest tokens over a paged cache, against 64-bit forms of its formula."""
import pytest
import torch

from fp8_implicit_gemm_gb300 import capi, q8
from _attention_common import CODE_ARG, CODES, attention64, check_attention, fill_cache, randn, values64

pytestmark = pytest.mark.gpu
WEIGHT_ROUND = 2.0 ** -11
TYPES = [torch.bfloat16, torch.float16]


def problem(codes, lengths, tokens, heads, kv, dim, page, dtype, seed=1, spread=1.0, extra_width=1, q_spread=2.0):
    width = max(1, -(-max(lengths + [1]) // page)) + extra_width
    cache = q8.CacheQ8.empty(len(lengths) * width + 1, page, kv, dim, CODE_ARG[codes])
    fill_cache(cache, codes, seed, spread)
    g = torch.Generator(device="cuda").manual_seed(seed)
    table = torch.randperm(cache.pages, generator=g, device="cuda")[:len(lengths) * width].view(-1, width).int()
    q = (randn(len(lengths) * tokens, heads, dim, seed=seed + 9) * q_spread).to(dtype)
    return cache, table, torch.tensor(lengths, dtype=torch.int32, device="cuda"), q


def verify(o, cache, codes, table, lengths, q, tokens, scale, what=""):
    k64, v64 = values64(cache, "k", codes), values64(cache, "v", codes)
    for b, n in enumerate(lengths.tolist()):
        pages = table[b].long()
        k, v = [x[pages].transpose(1, 2).flatten(0, 1)[:n] for x in (k64, v64)]
        limits = (n - tokens + 1 + torch.arange(tokens, device="cuda")).clamp(min=0)
        rows = slice(b * tokens, (b + 1) * tokens)
        want, size, worst = attention64(q[rows], k, v, limits, scale)
        check_attention(o[rows], want, size, worst, WEIGHT_ROUND, n, f"{what} sequence {b} of {n}")


def run(codes, lengths, tokens, heads, kv, dim, page, dtype, scale=None, **kw):
    cache, table, n, q = problem(codes, lengths, tokens, heads, kv, dim, page, dtype, **kw)
    attend = q8.CacheAttention(cache, heads, max_seqs=len(lengths), max_tokens=tokens, scale=scale)
    o = attend(q, table, n, torch.full_like(q, 7.0))
    assert attend.check() == capi.CONV3D_OK
    verify(o, cache, codes, table, n, q, tokens, dim ** -0.5 if scale is None else scale)
    attend.close()


@pytest.mark.parametrize("codes", CODES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 31, 63, 64, 65, 100, 257, 1000, 4099])
def test_lengths(codes, dtype, length):
    run(codes, [length], 1, 8, 2, 128, 16, dtype)


@pytest.mark.parametrize("codes", CODES)
@pytest.mark.parametrize("heads,kv", [(1, 1), (3, 1), (8, 8), (7, 1), (9, 1), (16, 1), (17, 1), (40, 1), (28, 4), (64, 8)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_heads(codes, heads, kv, dim):
    run(codes, [333, 40], 1, heads, kv, dim, 32, torch.bfloat16)


@pytest.mark.parametrize("codes", CODES)
@pytest.mark.parametrize("tokens", [1, 2, 3, 5, 8, 64])
def test_several_newest_tokens(codes, tokens):
    """Each sees one key more than the one before; sequences shorter than the tokens leave the first ones nothing."""
    run(codes, [tokens, 1, 700, 130, 0, 64 + tokens], tokens, 6, 2, 64, 48, torch.float16)


@pytest.mark.parametrize("codes", CODES)
@pytest.mark.parametrize("page", [16, 48, 64, 80, 256, 4096])
def test_ragged_batch(codes, page):
    g = torch.Generator().manual_seed(page)
    lengths = torch.randint(0, 3000, (40,), generator=g).tolist() + [0, 1, page, page + 1]
    run(codes, lengths, 1, 8, 2, 128, page, torch.bfloat16)


@pytest.mark.parametrize("codes", CODES)
def test_one_long_sequence(codes):
    run(codes, [50001], 1, 8, 1, 128, 64, torch.bfloat16)
    run(codes, [40000, 3], 2, 4, 2, 256, 128, torch.float16)


@pytest.mark.parametrize("codes", CODES)
def test_many_short_sequences(codes):
    run(codes, [i % 37 for i in range(700)], 1, 4, 2, 64, 16, torch.bfloat16)


@pytest.mark.parametrize("codes", CODES)
@pytest.mark.parametrize("q_spread,spread", [(40.0, 1.0), (1e-3, 1.0), (2.0, 1e-4), (2.0, 300.0), (0.0, 1.0)])
def test_sizes_of_values(codes, q_spread, spread):
    """One key that takes all the weight, equal weights, small and large values."""
    run(codes, [900], 1, 8, 2, 128, 16, torch.bfloat16, q_spread=q_spread, spread=spread)


@pytest.mark.parametrize("codes", CODES)
def test_scale(codes):
    for scale in (0.0, -0.1, 1.0):
        run(codes, [300], 1, 8, 2, 64, 16, torch.float16, scale=scale, q_spread=0.5)


@pytest.mark.parametrize("codes", CODES)
def test_v_scales_of_any_size(codes):
    """Rows of v whose scales differ by many powers of two, the largest ones with next to no weight."""
    cache, table, n, q = problem(codes, [500], 1, 4, 1, 64, 16, torch.bfloat16)
    g = torch.Generator(device="cuda").manual_seed(4)
    power = torch.randint(-20, 21, cache.v_scale.shape[:3], generator=g, device="cuda").float()
    cache.v_scale.mul_(torch.exp2(power) if codes != "i4" else torch.exp2(power)[..., None])
    attend = q8.CacheAttention(cache, 4)
    o = attend(q, table, n, torch.empty_like(q))
    verify(o, cache, codes, table, n, q, 1, 0.125)


@pytest.mark.parametrize("codes", CODES)
def test_what_lies_behind_a_sequence_is_not_used(codes):
    """Codes, scales and pages behind the end: NaN, infinities and page numbers out of range."""
    cache, table, n, q = problem(codes, [37, 100, 1], 1, 4, 1, 64, 16, torch.bfloat16, extra_width=2)
    attend = q8.CacheAttention(cache, 4, max_seqs=3)
    want = attend(q, table, n, torch.empty_like(q)).clone()
    used = torch.zeros(cache.pages, 16, dtype=torch.bool, device="cuda")
    for b, length in enumerate(n.tolist()):
        s = torch.arange(length, device="cuda")
        used[table[b].long()[s // 16], s % 16] = True
        table[b, -(-length // 16):] = -5 if b else 1 << 30
    for t in (cache.k_scale, cache.v_scale):
        t.masked_fill_((~used)[:, None, :].expand(t.shape[:3]) if t.dim() == 3 else (~used)[:, None, :, None].expand(t.shape),
                       float("nan"))
    for t in (cache.k_codes.view(torch.uint8), cache.v_codes.view(torch.uint8)):
        t.masked_fill_((~used)[:, None, :, None].expand(t.shape), 0x7F)  # NaN in e4m3
    o = attend(q, table, n, torch.empty_like(q))
    assert attend.check() == capi.CONV3D_OK
    assert torch.equal(o, want)
    for t in (cache.k_scale, cache.v_scale):
        t.masked_fill_(torch.isnan(t), float("inf"))
    assert torch.equal(attend(q, table, n, torch.empty_like(q)), want)


@pytest.mark.parametrize("codes", CODES)
@pytest.mark.parametrize("name", ["k", "v"])
def test_a_row_marked_nan_reaches_those_that_see_it(codes, name):
    cache, table, n, q = problem(codes, [60, 60], 3, 4, 2, 64, 16, torch.bfloat16)
    t = getattr(cache, name + "_scale")
    t.view(t.shape[:3] + (-1,))[table[0, 58 // 16].long(), 1, 58 % 16, 0] = float("nan")  # place 58, head 1
    attend = q8.CacheAttention(cache, 4, max_seqs=2, max_tokens=3)
    o = attend(q, table, n, torch.empty_like(q))
    assert attend.check() == capi.CONV3D_OK
    bad = torch.isnan(o)
    assert bool(bad[1:3, 2:].all()) and int(bad.sum()) == 2 * 2 * 64


@pytest.mark.parametrize("codes", CODES)
def test_bad_lengths_and_pages_are_reported(codes):
    cache, table, n, q = problem(codes, [60, 60, 60, 700], 1, 4, 2, 64, 16, torch.bfloat16, extra_width=0)
    attend = q8.CacheAttention(cache, 4, max_seqs=4)
    want = attend(q, table, n, torch.empty_like(q)).clone()
    assert attend.check() == capi.CONV3D_OK
    n[0], n[1] = -1, table.shape[1] * 16 + 1
    table[3, 20] = cache.pages
    o = attend(q, table, n, torch.empty_like(q))
    assert attend.check() == capi.CONV3D_EDEVICE
    assert attend.check() == capi.CONV3D_OK
    assert bool(torch.isnan(o[[0, 1, 3]]).all()) and torch.equal(o[2], want[2])
    n[0], n[1], table[3, 20] = 60, 60, -1
    o = attend(q, table, n, torch.empty_like(q))
    assert attend.check() == capi.CONV3D_EDEVICE
    assert bool(torch.isnan(o[3]).all()) and torch.equal(o[:3], want[:3])
    table[3, 20] = 0  # the plan goes on
    attend(q, table, n, o)
    assert attend.check() == capi.CONV3D_OK and bool(torch.isfinite(o).all())


def test_views_in_place_and_guards():
    cache, table, n, _ = problem("i8", [70, 5], 1, 4, 2, 64, 16, torch.bfloat16)
    full = randn(2, 12, 64, dtype=torch.bfloat16, seed=3)
    before = full.clone()
    q = full[:, 3:11:2]
    attend = q8.CacheAttention(cache, 4, max_seqs=2)
    want = attend(q.contiguous(), table, n, torch.empty(2, 4, 64, dtype=q.dtype, device="cuda"))
    out = torch.full((6, 2, 72), 7.0, dtype=torch.bfloat16, device="cuda")  # head first
    attend(q, table, n, out[1:5, :, :64].transpose(0, 1))
    assert torch.equal(out[1:5, :, :64].transpose(0, 1), want)
    out[1:5, :, :64] = 7.0
    assert bool((out == 7.0).all())
    attend(q, table, n, q)
    assert torch.equal(q, want)
    q.copy_(before[:, 3:11:2])
    assert torch.equal(full, before)
    wide = torch.zeros(2, table.shape[1] + 5, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    assert torch.equal(attend(q, wide[:, :table.shape[1]], n, torch.empty_like(want)), want)


def test_results_repeat_bit_by_bit():
    cache, table, n, q = problem("i4", [5000, 31, 999, 12000], 1, 32, 4, 128, 64, torch.bfloat16)
    attend = q8.CacheAttention(cache, 32, max_seqs=4)
    want = attend(q, table, n, torch.empty_like(q)).clone()
    for _ in range(20):
        assert torch.equal(attend(q, table, n, torch.empty_like(q)), want)


def test_fewer_sequences_and_tokens_than_planned_and_none():
    cache, table, n, q = problem("i8", [100, 900, 3], 2, 4, 2, 64, 16, torch.float16)
    attend = q8.CacheAttention(cache, 4, max_seqs=9, max_tokens=4)
    o = attend(q[:2], table[:1], n[:1], torch.empty_like(q[:2]))
    verify(o, cache, "i8", table[:1], n[:1], q[:2], 2, 0.125)
    o = attend(q[:3], table, n, torch.empty_like(q[:3]))
    verify(o, cache, "i8", table, n, q[:3], 1, 0.125)
    attend(q[:0], table[:0], n[:0], q[:0])
    assert attend.check() == capi.CONV3D_OK


def test_captured_replayed_with_other_lengths_and_on_other_streams():
    cache, table, n, q = problem("i4", [100, 6000, 3], 1, 8, 2, 128, 16, torch.bfloat16)
    attend = q8.CacheAttention(cache, 8, max_seqs=3)
    o = torch.empty_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        attend(q, table, n, o)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            attend(q, table, n, o)
        h = torch.cuda.CUDAGraph()
        with torch.cuda.graph(h, stream=s):
            attend(q, table, n, o)
    for lengths in ([100, 6000, 3], [6016, 1, 0], [64, 65, 3000]):
        n.copy_(torch.tensor(lengths, dtype=torch.int32))
        for graph in (g, h):
            o.fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            verify(o, cache, "i4", table, n, q, 1, 128 ** -0.5)
    assert attend.check() == capi.CONV3D_OK


def test_two_plans_at_once():
    cache, table, n, q = problem("i8", [9000, 100], 1, 8, 2, 128, 16, torch.bfloat16)
    plans = [q8.CacheAttention(cache, 8, max_seqs=2) for _ in range(2)]
    want = plans[0](q, table, n, torch.empty_like(q)).clone()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], [torch.empty_like(q) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for plan, s, o in zip(plans, streams, outs):
            plan(q, table, n, o, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


def test_refusals():
    cache, table, n, q = problem("i8", [100], 1, 4, 2, 64, 16, torch.bfloat16)
    attend = q8.CacheAttention(cache, 4)
    o = torch.empty_like(q)
    for args in ((q.float(), table, n, o.float()), (q, table.long(), n, o), (q, table, n.long(), o), (q, table, n[:0], o),
                 (q[:, :, :32], table, n, o[:, :, :32]), (q, table, n, o.half()), (q[:, :3], table, n, o[:, :3]),
                 (q.cpu(), table, n, o), (q, table.cpu(), n, o)):
        with pytest.raises((ValueError, capi.Conv3dFp8Error)):
            attend(*args)
    off = torch.empty(q.numel() + 1, dtype=q.dtype, device="cuda")[1:].view(q.shape)
    with pytest.raises(capi.Conv3dFp8Error):
        attend(off, table, n, o)
    with pytest.raises(capi.Conv3dFp8Error):
        attend(torch.cat([q, q]), table, n, torch.cat([o, o]))  # two tokens, planned for one


@pytest.mark.parametrize("codes", CODES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("b", [2.0 ** 11, 2.0 ** 13, 2.0 ** 15, 2.0 ** 30, 2.0 ** 95])
def test_scores_far_apart(codes, dtype, sign, b):
    """Key j scores sign * b * (j + 1) * 2^13 or more, so the last one has all the weight, or the first: the output is its
    value, off by its rounding to 16 bits and a few steps of fp32 of what the value is made of."""
    lengths, kv, dim = [1, 16, 100, 900], 2, 64
    cache, table, n, q = problem(codes, lengths, 1, 4, kv, dim, 16, dtype)
    q.zero_()
    q[..., 0] = sign * 2.0 ** 15
    one = {"i4": 0x01, "i8": 0x01, "e4m3": 0x38}[codes]
    cache.k_codes.view(torch.uint8).zero_()
    cache.k_codes.view(torch.uint8)[..., 0] = one
    for t, length in zip(table, lengths):
        at = torch.arange(t.numel() * 16, device="cuda").view(-1, 1, 16).expand(-1, kv, -1)
        scale = b * (at + 1).float()
        cache.k_scale[t.long()] = torch.stack([scale, torch.zeros_like(scale)], dim=-1) if codes == "i4" else scale
    attend = q8.CacheAttention(cache, 4, max_seqs=4)
    o = attend(q, table, n, torch.full_like(q, 7.0))
    assert attend.check() == capi.CONV3D_OK
    v64 = values64(cache, "v", codes)
    for i, length in enumerate(lengths):
        at = length - 1 if sign > 0 else 0
        want = v64[int(table[i, at // 16]), :, at % 16].repeat_interleave(2, dim=0)
        size = cache.v_scale[int(table[i, at // 16]), :, at % 16].double().abs().reshape(kv, -1)
        size = (size[:, 0] * (16 if codes == "i4" else 1) + size[:, -1]).repeat_interleave(2)[:, None]
        bound = want.abs() * torch.finfo(dtype).eps / 2 + (want.abs() + size) * 2.0 ** -20 + torch.finfo(dtype).smallest_normal * 2.0 ** -10
        assert bool(((o[i].double() - want).abs() <= bound).all()), length
