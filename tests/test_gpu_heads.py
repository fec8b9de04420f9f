"""Norms and rotations of heads, caches of codes and their reading, against 64-bit forms of their formulas."""
import pytest
import torch

from fp8_implicit_gemm_gb300 import capi, q8
from _attention_common import (CODE_ARG, CODES, ROUND, TINY, U, codes64, fill_cache, heads64, randn, unpack,
                               values64)

pytestmark = pytest.mark.gpu
EPS = 1e-6
TYPES = [torch.bfloat16, torch.float16, torch.float32]
ERR = 2.0 ** -19


def frequencies(sections, theta=10000.0):
    return torch.cat([theta ** -(torch.arange(n, dtype=torch.float64) / n) for n in sections]).cuda()


def check(got, want, size, err=ERR):
    r, tiny = ROUND[got.dtype], TINY[got.dtype]
    e = err * size + 2.0 ** -140
    off = (got.double() - want).abs() - ((e + (want.abs() + e) * r) * (1 + 2.0 ** -20) + tiny)
    assert bool(torch.isfinite(got).all())
    assert off.numel() == 0 or float(off.max()) <= 0.0, float(off.max())


def guarded(tokens, heads, dim, dtype, head_first=False):
    """A view inside a larger matrix of a known filling."""
    shape = (heads, tokens + 2, dim + 16) if head_first else (tokens, heads + 2, dim + 16)
    full = torch.full(shape, 7.0, dtype=dtype, device="cuda")
    if head_first:
        return full[:, 1:1 + tokens, 8:8 + dim].transpose(0, 1), full
    return full[:, 1:1 + heads, 8:8 + dim], full


def untouched(full, view):
    """Only the view's elements differ from the filling."""
    keep = full.clone()
    view.fill_(7.0)
    assert bool((full == 7.0).all())
    full.copy_(keep)


# tokens, q heads, k heads, dim, rot, sections, adjacent, norm
CASES = [(1, 1, 1, 8, 8, [4], False, True), (3, 2, 1, 8, 2, [1], True, True), (1, 32, 8, 128, 128, [64], False, True),
         (5, 4, 2, 64, 64, [32], True, False), (7, 3, 3, 80, 40, [20], False, True), (33, 2, 1, 96, 96, [16, 16, 16], True, True),
         (17, 5, 1, 256, 256, [32, 48, 48], False, True), (40, 1, 1, 72, 72, [18, 18], False, False),
         (300, 16, 4, 128, 64, [32], False, True), (1000, 2, 2, 128, 128, [16, 24, 24], True, True),
         (9, 1, 1, 16, 6, [3], False, True), (64, 1, 3, 112, 112, [14, 14, 14, 14], False, True),
         (2, 60, 60, 256, 100, [50], False, False), (611, 7, 1, 40, 0, None, False, True)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case", CASES, ids=str)
def test_heads(dtype, case):
    tokens, heads, kv, dim, rot, sections, adjacent, norm = case
    q, k = randn(tokens, heads, dim, dtype=dtype, seed=1), randn(tokens, kv, dim, dtype=dtype, seed=2)
    qw, kw = [(1 + 0.1 * randn(dim, seed=s)).to(dtype if s == 3 else dtype) for s in (3, 4)] if norm else (None, None)
    rotary = positions = freqs = axis = None
    if rot:
        rotary = q8.Rotary(rot, sections=sections, adjacent=adjacent)
        freqs = frequencies(sections)
        axis = torch.repeat_interleave(torch.arange(len(sections)), torch.tensor(sections)).cuda()
        g = torch.Generator(device="cuda").manual_seed(5)
        positions = torch.randint(-50, 200000, (len(sections), tokens), generator=g, device="cuda")
    (qo, q_full), (ko, k_full) = guarded(tokens, heads, dim, dtype), guarded(tokens, kv, dim, dtype, True)
    capi.heads_q8_run(q=q, q_out=qo, k=k, k_out=ko, q_weight=qw, k_weight=kw, eps=EPS, rotary=rotary,
                      positions=positions)
    check(qo, *heads64(q, qw, EPS, freqs, axis, positions, rot, adjacent))
    check(ko, *heads64(k, kw, EPS, freqs, axis, positions, rot, adjacent))
    untouched(q_full, qo)
    untouched(k_full, ko)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rot,adjacent", [(64, False), (40, False), (64, True)])
def test_heads_in_place_of_one_matrix(dtype, rot, adjacent):
    """As a product leaves q, k and v: views of one matrix, turned where they lie."""
    x = randn(37, 10, 64, dtype=dtype, seed=1)
    before = x.clone()
    rotary, freqs = q8.Rotary(rot, adjacent=adjacent), frequencies([rot // 2])
    pos = torch.arange(37, device="cuda") * 3000
    w = randn(64, dtype=torch.float32, seed=2)
    capi.heads_q8_run(q=x[:, :6], q_out=x[:, :6], k=x[:, 6:8], k_out=x[:, 6:8], q_weight=w, rotary=rotary, positions=pos)
    axis = torch.zeros(rot // 2, dtype=torch.int64, device="cuda")
    check(x[:, :6], *heads64(before[:, :6], w, EPS, freqs, axis, pos[None], rot, adjacent))
    check(x[:, 6:8], *heads64(before[:, 6:8], None, EPS, freqs, axis, pos[None], rot, adjacent))
    assert torch.equal(x[:, 8:], before[:, 8:])


def test_only_queries_or_only_keys():
    x, out = randn(5, 3, 64, seed=1), torch.empty(5, 3, 64, device="cuda")
    rotary, pos = q8.Rotary(64), torch.arange(5, device="cuda")
    axis, freqs = torch.zeros(32, dtype=torch.int64, device="cuda"), frequencies([32])
    want = heads64(x, None, EPS, freqs, axis, pos[None], 64)
    capi.heads_q8_run(q=x, q_out=out, rotary=rotary, positions=pos)
    check(out, *want)
    out.zero_()
    capi.heads_q8_run(k=x, k_out=out, rotary=rotary, positions=pos)
    check(out, *want)


def test_far_positions():
    """The fraction of a turn is exact: turned by a position p and by p modulo the exact period agree."""
    import math
    freqs = [2 * math.pi * 2.0 ** -20, 2 * math.pi * 3 * 2.0 ** -24, 1e-3, 1.0]
    rotary = q8.Rotary(8, frequencies=freqs)
    x = randn(4, 1, 8, seed=1)
    near = torch.tensor([5, 77, 0, 123456], device="cuda")
    far = near + (1 << 40)  # whole periods of the first two pairs
    a, b = torch.empty_like(x), torch.empty_like(x)
    capi.heads_q8_run(q=x, q_out=a, rotary=rotary, positions=near)
    capi.heads_q8_run(q=x, q_out=b, rotary=rotary, positions=far)
    assert torch.equal(a[..., [0, 1, 4, 5]], b[..., [0, 1, 4, 5]])
    import fractions
    turns = [fractions.Fraction(t % 2 ** 64, 2 ** 64) for t in rotary._turns.tolist()]
    for i, p in enumerate(far.tolist()):
        for j in range(4):
            angle = 2 * math.pi * float(turns[j] * p % 1)
            u, v = float(x[i, 0, j]), float(x[i, 0, j + 4])
            assert abs(float(b[i, 0, j]) - (u * math.cos(angle) - v * math.sin(angle))) <= 2 ** -19 * (abs(u) + abs(v))


@pytest.mark.parametrize("size", [2.0 ** -149, 1e-44, 1e-38, 1e-25, 1e-13, 1e13, 1e25, 3e38])
def test_tiny_and_huge_rows_are_normed(size):
    """With an eps of 0 the norm does not depend on the row's size (eighths of it are exact in fp32 from 2^-146 on; the
    form takes the rounded values)."""
    x = (torch.tensor([[[1.0, -0.5, 0.25, 0.0, 0.75, -1.0, 0.125, 0.5]]], device="cuda").double() * size).float()
    w, out = torch.ones(8, device="cuda"), torch.empty_like(x)
    capi.heads_q8_run(q=x, q_out=out, q_weight=w, eps=0.0)
    check(out, *heads64(x, w, 0.0))
    capi.heads_q8_run(q=x, q_out=out, q_weight=w, eps=1.0)
    check(out, *heads64(x, w, 1.0))


def test_rows_of_zeros_and_bad_rows():
    x = randn(6, 2, 64, dtype=torch.bfloat16, seed=1)
    x[1] = 0
    x[2, 0, 5], x[3, 1, 7] = float("nan"), float("inf")
    w, out = torch.ones(64, dtype=torch.bfloat16, device="cuda"), torch.empty_like(x)
    capi.heads_q8_run(q=x, q_out=out, q_weight=w, eps=0.0)
    assert float(out[1].abs().max()) == 0.0
    assert bool(torch.isnan(out[2, 0]).all()) and bool(torch.isnan(out[3, 1, 7]))
    assert bool(torch.isfinite(out[[0, 4, 5]]).all() and torch.isfinite(out[2, 1]).all() and torch.isfinite(out[3, 0]).all())


def test_weights_of_every_type():
    x = randn(3, 2, 64, dtype=torch.bfloat16, seed=1)
    for wt in TYPES:
        w, out = randn(65, dtype=wt, seed=2)[1:], torch.empty_like(x)
        capi.heads_q8_run(q=x, q_out=out, q_weight=w)
        check(out, *heads64(x, w))


# ------------------------------------------------------------------------------------- the cache
def slots_of(tokens, cache, seed, page_order=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randperm(cache.pages * cache.page_size, generator=g, device="cuda")[:tokens]


def rows_at(t, slots, page_size):
    return t[slots // page_size, :, slots % page_size]


@pytest.mark.parametrize("codes", CODES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,kv,dim,page", [(1, 1, 64, 16), (5, 3, 128, 16), (100, 2, 256, 48), (333, 5, 64, 32),
                                                (2000, 1, 128, 256)])
def test_write_and_read(codes, dtype, tokens, kv, dim, page):
    cache = q8.CacheQ8.empty(-(-tokens // page) + 2, page, kv, dim, CODE_ARG[codes])
    cache.k_codes.view(torch.uint8).fill_(0x55), cache.v_codes.view(torch.uint8).fill_(0x55)
    cache.k_scale.fill_(-3.0), cache.v_scale.fill_(-3.0)
    k, v = randn(tokens, kv, dim, dtype=dtype, seed=1), randn(tokens, kv, dim, dtype=dtype, seed=2)
    k[0] = 0.5
    v[-1] = 0.0
    slots = slots_of(tokens, cache, 3)
    slots[tokens // 2] = -1 if tokens % 2 else cache.pages * page
    live = torch.arange(tokens, device="cuda") != tokens // 2
    capi.heads_q8_run(k=k, v=v, cache=cache, slots=slots)
    for name, x in (("k", k), ("v", v)):
        q, scale, lowest = codes64(x, codes)
        got = unpack(rows_at(getattr(cache, name + "_codes").view(torch.uint8), slots[live], page)
                     .view(cache.k_codes.dtype), codes)
        s = rows_at(getattr(cache, name + "_scale"), slots[live], page)
        if codes == "i4":
            assert torch.equal(s[..., 1].double(), lowest[live])
            s = s[..., 0]
        assert bool(((s.double() - scale[live]).abs() <= 2 * U * scale[live]).all())
        if dtype != torch.float32:  # quotients of 16-bit values are decided exactly
            assert torch.equal(got, q[live])
        else:
            # a quotient of fp32 values errs by u of itself, and where that is next to a tie by a step
            step = 1.0 if codes != "e4m3" else torch.exp2(torch.frexp(q.abs().clamp(min=2.0 ** -6))[1].double() - 4)[live]
            assert bool(((got - q[live]).abs() <= step * 1.0001).all())
            assert int((got != q[live]).sum()) <= 1e-4 * got.numel()
    taken = torch.zeros(cache.pages * page, dtype=torch.bool, device="cuda")
    taken[slots[live]] = True
    rest = (~taken).nonzero()[:, 0]
    assert bool((rows_at(cache.k_codes.view(torch.uint8), rest, page) == 0x55).all())
    assert bool((rows_at(cache.v_scale, rest, page) == -3.0).all())
    # and back, into a view with gaps; rows of padding slots stay
    (ko, k_full), (vo, v_full) = guarded(tokens, kv, dim, dtype), guarded(tokens, kv, dim, dtype, True)
    cache.read(slots, ko, vo)
    for name, out in (("k", ko), ("v", vo)):
        want = rows_at(values64(cache, name, codes), slots[live], page)
        size = want.abs() + (rows_at(getattr(cache, name + "_scale"), slots[live], page)[..., 1:].double().abs()
                             if codes == "i4" else 0)
        check(out[live], want, size, 2 * U)
        assert bool((out[~live] == 7.0).all())
    untouched(k_full, ko)
    untouched(v_full, vo)


@pytest.mark.parametrize("codes", CODES)
def test_normed_and_turned_keys_into_the_cache(codes):
    """In one call: q to its output, k normed, turned and as codes of the unrounded values (k_out beside them), v as it
    is. The code of a value that errs by 2^-19 of the row's size is off by that much of the code's range and half a step."""
    tokens, heads, kv, dim, page = 70, 8, 2, 128, 16
    x = randn(tokens, heads + 2 * kv, dim, dtype=torch.bfloat16, seed=1)
    w = (1 + 0.1 * randn(2, dim, seed=2)).bfloat16()
    rotary, freqs = q8.Rotary(dim), frequencies([dim // 2])
    pos, axis = torch.arange(tokens, device="cuda") + 70000, torch.zeros(dim // 2, dtype=torch.int64, device="cuda")
    cache = q8.CacheQ8.empty(9, page, kv, dim, CODE_ARG[codes])
    slots = slots_of(tokens, cache, 3)
    q_out, k_out = torch.empty(tokens, heads, dim, dtype=x.dtype, device="cuda"), torch.empty(tokens, kv, dim, dtype=x.dtype, device="cuda")
    capi.heads_q8_run(q=x[:, :heads], q_out=q_out, k=x[:, heads:-kv], k_out=k_out, v=x[:, -kv:], q_weight=w[0],
                      k_weight=w[1], rotary=rotary, positions=pos, cache=cache, slots=slots)
    check(q_out, *heads64(x[:, :heads], w[0], EPS, freqs, axis, pos[None], dim))
    k, size = heads64(x[:, heads:-kv], w[1], EPS, freqs, axis, pos[None], dim)
    check(k_out, k, size)
    got = rows_at(values64(cache, "k", codes), slots, page)
    amax = k.abs().amax(-1, keepdim=True)
    step = {"i8": amax / 127, "i4": (k.amax(-1, keepdim=True) - k.amin(-1, keepdim=True)) / 15,
            "e4m3": torch.maximum(k.abs() * 2.0 ** -3 * 1.01, amax / 448 * 2.0 ** -9)}[codes]
    assert bool(((got - k).abs() <= step / 2 * (1 + 2.0 ** -10) + 2 * ERR * size.amax(-1, keepdim=True)).all())
    got = rows_at(values64(cache, "v", codes), slots, page)
    q, scale, lowest = codes64(x[:, -kv:], codes)
    assert bool(((got - (q * scale[..., None] + (lowest[..., None] if codes == "i4" else 0))).abs() <= 4 * U * (
        x[:, -kv:].double().abs().amax(-1, keepdim=True)) * 2).all())


@pytest.mark.parametrize("codes", CODES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_rows_that_are_not_finite(codes, bad):
    cache = q8.CacheQ8.empty(2, 16, 2, 64, CODE_ARG[codes])
    k, v = randn(4, 2, 64, dtype=torch.bfloat16, seed=1), randn(4, 2, 64, dtype=torch.bfloat16, seed=2)
    k[1, 0, 3], v[2, 1, 60] = bad, bad
    slots = torch.tensor([3, 17, 4, 20], device="cuda")
    capi.heads_q8_run(k=k, v=v, cache=cache, slots=slots)
    ks, vs = [rows_at(s, slots, 16).reshape(4, 2, -1)[..., 0] for s in (cache.k_scale, cache.v_scale)]
    assert bool(torch.isnan(ks[1, 0])) and bool(torch.isnan(vs[2, 1]))
    assert int(torch.isnan(ks).sum()) == int(torch.isnan(vs).sum()) == 1
    assert bool((rows_at(cache.k_codes.view(torch.uint8), slots, 16)[1, 0] == 0).all())
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    cache.read(slots, ko, vo)
    assert bool(torch.isnan(ko[1, 0]).all()) and bool(torch.isnan(vo[2, 1]).all())
    assert int(torch.isnan(ko).sum()) == int(torch.isnan(vo).sum()) == 64


@pytest.mark.parametrize("codes", CODES)
@pytest.mark.parametrize("size", [2.0 ** -149, 2.0 ** -140, 2.0 ** -126, 2.0 ** -101, 2.0 ** 101, 2.0 ** 125])
def test_codes_of_tiny_and_huge_rows(codes, size):
    """The codes are those of the exact quotient even where the scale is coarse or 0."""
    v = torch.tensor([1.0, -0.5, 0.25, 0.0] * 16, device="cuda").double()[None, None] * size
    x = v.float()
    cache = q8.CacheQ8.empty(1, 16, 1, 64, CODE_ARG[codes])
    capi.heads_q8_run(k=x, v=x, cache=cache, slots=torch.tensor([7], device="cuda"))
    q, scale, lowest = codes64(x, codes)
    assert torch.equal(unpack(cache.k_codes, codes)[0, 0, 7], q[0, 0])
    s = cache.k_scale.view(1, 1, 16, -1)[0, 0, 7]
    assert abs(float(s[0]) - float(scale)) <= 2 * U * float(scale) + 2.0 ** -150


def test_a_range_past_fp32_marks_the_row():
    x = torch.zeros(1, 1, 64, device="cuda")
    x[0, 0, 0], x[0, 0, 1] = 3e38, -3e38
    cache = q8.CacheQ8.empty(1, 16, 1, 64, 4)
    capi.heads_q8_run(k=x, v=x, cache=cache, slots=torch.tensor([0], device="cuda"))
    assert bool(torch.isnan(cache.k_scale[0, 0, 0, 0])) and int(cache.k_codes.max()) == 0


def test_one_slot_read_twice_and_no_tokens():
    cache = q8.CacheQ8.empty(2, 16, 3, 64, torch.int8)
    fill_cache(cache, "i8", 1)
    slots = torch.tensor([5, 5, 31, -7, 32, 1 << 40], device="cuda")
    k, v = torch.full((2, 6, 3, 64), 7.0, device="cuda")
    cache.read(slots, k, v)
    assert torch.equal(k[0], k[1]) and bool((k[3:] == 7.0).all()) and bool((v[3:] == 7.0).all())
    none = torch.empty(0, 3, 64, device="cuda")
    cache.read(slots[:0], none, none)
    capi.heads_q8_run(k=none, v=none, cache=cache, slots=slots[:0])
    capi.heads_q8_run(q=none, q_out=none)


def test_large_cache_offsets():
    """Codes past 2^32 bytes: the last pages of a cache of 5 GB."""
    pages, page, kv, dim = 20000, 256, 4, 256
    cache = q8.CacheQ8.empty(pages, page, kv, dim, torch.int8)
    k, v = randn(3, kv, dim, dtype=torch.bfloat16, seed=1), randn(3, kv, dim, dtype=torch.bfloat16, seed=2)
    slots = torch.tensor([pages * page - 1, (pages - 3) * page, 17], device="cuda")
    capi.heads_q8_run(k=k, v=v, cache=cache, slots=slots)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    cache.read(slots, ko, vo)
    for got, x in ((ko, k), (vo, v)):
        q, scale, _ = codes64(x, "i8")
        check(got, q * scale[..., None], q.abs() * scale[..., None], 4 * U)
    assert int((cache.k_codes[pages - 2:, :, :page - 1] != 0).sum()) == 0


def test_captured_and_replayed():
    cache = q8.CacheQ8.empty(4, 16, 2, 64, 4)
    x = randn(10, 8, 64, dtype=torch.bfloat16, seed=1)
    q_out, back = torch.empty(10, 4, 64, dtype=x.dtype, device="cuda"), torch.empty(2, 10, 2, 64, dtype=x.dtype, device="cuda")
    slots, rotary, pos = torch.arange(10, device="cuda") * 5, q8.Rotary(64), torch.arange(10, device="cuda")

    def step():
        capi.heads_q8_run(q=x[:, :4], q_out=q_out, k=x[:, 4:6], v=x[:, 6:], rotary=rotary, positions=pos, cache=cache, slots=slots)
        cache.read(slots, back[0], back[1])
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step()
    for seed in (5, 6):
        x.copy_(randn(10, 8, 64, dtype=torch.bfloat16, seed=seed))
        pos.add_(1000)
        g.replay()
        torch.cuda.synchronize()
        got = q_out.clone(), back.clone()
        step()
        assert torch.equal(got[0], q_out) and torch.equal(got[1], back)
