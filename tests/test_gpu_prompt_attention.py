"""Attention over whole prompts, against 64-bit forms of its formula."""
import pytest
import torch

from fp8_implicit_gemm_gb300 import capi, q8
from _attention_common import ROUND, attention64, check_attention, randn

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16]


def starts_of(lengths, first=0):
    return torch.tensor([first] + lengths, device="cuda").cumsum(0).int()


def verify(o, q, k, v, starts, key_starts, causal, scale, what=""):
    for b in range(starts.numel() - 1):
        a, e = int(starts[b]), int(starts[b + 1])
        c, d = int(key_starts[b]), int(key_starts[b + 1])
        n, m = e - a, d - c
        limits = torch.full((n,), m, device="cuda")
        if causal:
            limits = (torch.arange(1, n + 1, device="cuda") + m - n).clamp(min=0)
        for i in range(0, n, 512):  # the 64-bit weights of some rows at a time
            rows = slice(a + i, min(e, a + i + 512))
            want, size, worst = attention64(q[rows], k[c:d], v[c:d], limits[i:i + 512], scale)
            check_attention(o[rows], want, size, worst, ROUND[o.dtype], m, f"{what} sequence {b} from {i}")


def run(lengths, heads, kv, dim, dtype, causal=True, key_lengths=None, scale=None, seed=1, q_spread=2.0):
    rows, keys = sum(lengths), sum(key_lengths or lengths)
    q = (randn(rows, heads, dim, seed=seed) * q_spread).to(dtype)
    k, v = randn(keys, kv, dim, dtype=dtype, seed=seed + 1), randn(keys, kv, dim, dtype=dtype, seed=seed + 2)
    starts = starts_of(lengths)
    key_starts = starts_of(key_lengths) if key_lengths else None
    attend = q8.PromptAttention(scale=scale)
    o = attend(q, k, v, starts, torch.full_like(q, 7.0), causal=causal, key_starts=key_starts)
    assert attend.check() == capi.CONV3D_OK
    verify(o, q, k, v, starts, starts if key_starts is None else key_starts, causal,
           dim ** -0.5 if scale is None else scale)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("length", [1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 511, 513, 1000, 2049])
def test_lengths(dtype, causal, length):
    run([length], 2, 1, 128, dtype, causal)


@pytest.mark.parametrize("dim", [8, 16, 40, 64, 72, 80, 96, 112, 120, 128])
@pytest.mark.parametrize("heads,kv", [(1, 1), (4, 4), (7, 1), (6, 2)])
def test_heads(dim, heads, kv):
    run([140, 333], heads, kv, dim, torch.bfloat16, dim % 16 == 0)
    run([200], heads, kv, dim, torch.float16, True)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", TYPES)
def test_packed(causal, dtype):
    run([1, 0, 128, 300, 0, 0, 5, 777, 256, 2], 4, 2, 64, dtype, causal)
    run([3] * 200, 2, 1, 128, dtype, causal)


@pytest.mark.parametrize("causal", [True, False])
def test_chunks_of_queries(causal):
    """Queries whose keys begin earlier, fewer keys than queries (rows that see nothing), and no keys at all."""
    run([100, 1, 130, 300, 64, 7], 4, 2, 128, torch.bfloat16, causal, key_lengths=[1000, 513, 130, 90, 0, 64])


def test_long():
    run([9001], 2, 1, 128, torch.bfloat16)
    run([64], 4, 1, 64, torch.float16, True, key_lengths=[20000])


@pytest.mark.parametrize("q_spread,scale", [(40.0, None), (1e-3, None), (0.0, None), (1.0, 1.0), (1.0, -0.1), (3.0, 0.0)])
@pytest.mark.parametrize("dtype", TYPES)
def test_sizes_of_scores(q_spread, scale, dtype):
    run([500], 2, 1, 128, dtype, True, q_spread=q_spread, scale=scale)


def test_scores_that_grow_and_fall():
    """Later keys with ever larger scores, so that the running maximum moves all the time, and the reverse."""
    for order in (1, -1):
        n, dim = 700, 64
        q = torch.ones(n, 1, dim, device="cuda").bfloat16()
        k = torch.arange(n, device="cuda").float() if order > 0 else torch.arange(n - 1, -1, -1, device="cuda").float()
        k = (k[:, None, None] / 8).expand(n, 1, dim).contiguous().bfloat16()
        v = randn(n, 1, dim, dtype=torch.bfloat16, seed=1)
        starts = starts_of([n])
        o = q8.PromptAttention()(q, k, v, starts, torch.empty_like(q), causal=False)
        verify(o, q, k, v, starts, starts, False, dim ** -0.5)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("where", [0, 5, 100, 127, 128, 200, 299])
def test_what_a_row_does_not_see_does_not_reach_it(dtype, bad, where):
    """A key or value that is not finite: rows before it, and other sequences, are as without it."""
    lengths, dim = [300, 300], 64
    q = randn(600, 2, dim, dtype=dtype, seed=1)
    k, v = randn(600, 1, dim, dtype=dtype, seed=2), randn(600, 1, dim, dtype=dtype, seed=3)
    starts, attend = starts_of(lengths), q8.PromptAttention()
    want = attend(q, k, v, starts, torch.empty_like(q))
    for t, channel in ((k, 9), (v, 9)):
        keep = t[where, 0, channel].clone()
        t[where, 0, channel] = bad
        o = attend(q, k, v, starts, torch.empty_like(q))
        assert attend.check() == capi.CONV3D_OK
        assert torch.equal(o[:where], want[:where]) and torch.equal(o[300:], want[300:])
        if t is v:
            others = [c for c in range(dim) if c != channel]
            assert torch.equal(o[where:300][..., others], want[where:300][..., others])
            assert not bool(torch.isfinite(o[where:300][..., channel]).any())
        elif bad != bad:
            assert bool(torch.isnan(o[where:300]).all())
        # behind the end of the last sequence too
        t[where, 0, channel] = keep
        short = starts_of([where, 0])
        t[where:] = bad
        o = attend(q, k, v, short, torch.full_like(q, 7.0))
        assert torch.equal(o[:where], want[:where]) and bool((o[where:] == 7.0).all())
        t.copy_(randn(600, 1, dim, dtype=dtype, seed=2 if t is k else 3))


def test_a_query_that_is_not_finite_stays_alone():
    q = randn(300, 2, 128, dtype=torch.bfloat16, seed=1)
    k, v = randn(300, 1, 128, dtype=torch.bfloat16, seed=2), randn(300, 1, 128, dtype=torch.bfloat16, seed=3)
    starts, attend = starts_of([300]), q8.PromptAttention()
    want = attend(q, k, v, starts, torch.empty_like(q))
    q[77, 1, 5] = float("nan")
    o = attend(q, k, v, starts, torch.empty_like(q))
    assert bool(torch.isnan(o[77, 1]).all())
    o[77, 1] = want[77, 1]
    assert torch.equal(o, want)


def test_rows_outside_all_sequences_stay():
    q = randn(900, 2, 64, dtype=torch.float16, seed=1)
    k, v = randn(900, 2, 64, dtype=torch.float16, seed=2), randn(900, 2, 64, dtype=torch.float16, seed=3)
    starts = torch.tensor([100, 250, 251, 700], dtype=torch.int32, device="cuda")
    attend = q8.PromptAttention()
    o = attend(q, k, v, starts, torch.full_like(q, 7.0))
    verify(o, q, k, v, starts, starts, True, 0.125)
    assert bool((o[:100] == 7.0).all()) and bool((o[700:] == 7.0).all())


def test_bad_starts_are_cut():
    """Starts that decrease or leave the rows: nothing outside is read or written."""
    q = randn(300, 1, 64, dtype=torch.bfloat16, seed=1)
    k, v = randn(300, 1, 64, dtype=torch.bfloat16, seed=2), randn(300, 1, 64, dtype=torch.bfloat16, seed=3)
    attend = q8.PromptAttention()
    for starts, cut in (([-50, 100], [0, 100]), ([200, 1000], [200, 300]), ([50, 20], None), ([400, 500], None),
                        ([1 << 30, -(1 << 30)], None)):
        s = torch.tensor(starts, dtype=torch.int32, device="cuda")
        o = attend(q, k, v, s, torch.full_like(q, 7.0))
        assert attend.check() == capi.CONV3D_OK
        a, e = cut or (0, 0)
        s = torch.tensor([a, e], dtype=torch.int32, device="cuda")
        verify(o, q, k, v, s, s, True, 0.125)
        assert bool((o[:a] == 7.0).all()) and bool((o[e:] == 7.0).all())


@pytest.mark.parametrize("dtype", TYPES)
def test_views(dtype):
    """q, k and v as views of one matrix, with the output in a matrix with gaps; heads before tokens."""
    x = randn(333, 9, 72, dtype=dtype, seed=1)
    q, k, v = x[:, :4, :64], x[:, 4:6, 8:], x[:, 6:8, :64]
    full = torch.full((6, 335, 80), 7.0, dtype=dtype, device="cuda")
    o = full[1:5, 1:334, 8:72].transpose(0, 1)
    starts, attend = starts_of([200, 133]), q8.PromptAttention()
    attend(q, k, v, starts, o)
    verify(o, q, k, v, starts, starts, True, 0.125)
    want = attend(q.contiguous(), k.contiguous(), v.contiguous(), starts, torch.empty(333, 4, 64, dtype=dtype, device="cuda"))
    assert torch.equal(o, want)
    o.fill_(7.0)
    assert bool((full == 7.0).all())
    t = x.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(attend(t[:, :4, :64], t[:, 4:6, 8:], t[:, 6:8, :64], starts, torch.empty_like(want)), want)


def test_offsets_past_32_bits():
    """Heads 2^32 elements apart."""
    n, dim = 200, 64
    big = torch.empty((1 << 32) + n * dim, dtype=torch.bfloat16, device="cuda")
    k = big.as_strided((n, 2, dim), (dim, 1 << 32, 1))
    k.copy_(randn(n, 2, dim, dtype=torch.bfloat16, seed=2))
    q, v = randn(n, 2, dim, dtype=torch.bfloat16, seed=1), randn(n, 2, dim, dtype=torch.bfloat16, seed=3)
    starts = starts_of([n])
    o = q8.PromptAttention()(q, k, v, starts, torch.empty_like(q))
    verify(o, q, k.contiguous(), v, starts, starts, True, 0.125)


def test_captured_and_replayed_and_at_once():
    q = randn(700, 4, 128, dtype=torch.bfloat16, seed=1)
    k, v = randn(700, 2, 128, dtype=torch.bfloat16, seed=2), randn(700, 2, 128, dtype=torch.bfloat16, seed=3)
    starts, attend = starts_of([300, 400]), q8.PromptAttention()
    o = torch.empty_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        attend(q, k, v, starts, o)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            attend(q, k, v, starts, o)
    for cut in (300, 1, 699, 700):
        starts[1] = cut
        o.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        verify(o, q, k, v, starts, starts, True, 128 ** -0.5)
    want = o.clone()
    outs = [torch.empty_like(q) for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in outs]
    torch.cuda.synchronize()
    for _ in range(10):
        for t, st in zip(outs, streams):
            attend(q, k, v, starts, t, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(t, want) for t in outs)
    assert attend.check() == capi.CONV3D_OK


def test_none_and_refusals():
    q = randn(10, 2, 64, dtype=torch.bfloat16, seed=1)
    starts, attend = starts_of([10]), q8.PromptAttention()
    attend(q[:0], q[:0], q[:0], starts, q[:0])
    o = torch.full_like(q, 7.0)
    attend(q, q[:0], q[:0], starts, o, key_starts=torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert float(o.abs().max()) == 0.0
    attend(q, q, q, starts[:1], o)
    for args, kw in (((q.float(), q.float(), q.float(), starts, o.float()), {}), ((q, q, q, starts.long(), o), {}),
                     ((q, q[:5], q[:5], starts, o), {}), ((q, q, q.half(), starts, o), {}), ((q, q, q, starts.cpu(), o), {}),
                     ((q[:, :1], q, q, starts, o[:, :1]), {}), ((q, q, q, starts, o), dict(key_starts=starts[:1])),
                     ((q[..., :60], q[..., :60], q[..., :60], starts, o[..., :60]), {}),
                     ((q.cpu(), q, q, starts, o), {})):
        with pytest.raises((ValueError, capi.Conv3dFp8Error)):
            attend(*args, **kw)
    wide = randn(10, 2, 136, dtype=torch.bfloat16, seed=1)
    with pytest.raises(capi.Conv3dFp8Error):
        attend(wide, wide, wide, starts, torch.empty_like(wide))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,a,b", [(torch.float16, 6e4, 256.0), (torch.float16, -6e4, 256.0), (torch.float16, 6e4, 1.0),
                                       (torch.bfloat16, 1e16, 2.0 ** 48), (torch.bfloat16, -1e16, 2.0 ** 48),
                                       (torch.bfloat16, -1e16, 2.0 ** 58), (torch.bfloat16, 1e4, 2.0 ** 20)])
def test_scores_far_apart(dtype, a, b, causal):
    """Key j scores a * b * (j + 1) times a constant: the last visible one has all the weight, or the first where a < 0, the
    others less than 2^-1000 of it. So the output is that key's value v. Its weight p is rounded to the type beside v, by d of
    it, and not in the sum (p is a power of two only where its exponent is exact, which fp32 scores of up to 2^16 are not), then
    the output is rounded: with h = eps / 2, |d| <= h and fp32's steps in between of less than 2^-20, |o - v| <= |v| (h + 2^-20) (1 + h)
    + |v| h <= |v| eps (1 + 2^-7); and half a step of subnormal numbers."""
    rows, heads, dim = 200, 2, 64
    q, k = torch.zeros(2, rows, heads, dim, dtype=dtype, device="cuda")
    q[..., 0] = a
    k[..., 0] = (b * torch.arange(1, rows + 1, device="cuda", dtype=torch.float64)).to(dtype)[:, None]
    v = randn(rows, heads, dim, dtype=dtype, seed=3)
    attend = q8.PromptAttention()
    o = attend(q, k, v, starts_of([rows]), torch.empty_like(q), causal=causal)
    assert attend.check() == capi.CONV3D_OK
    want = (v[:1].expand_as(v) if a < 0 else v if causal else v[-1:].expand_as(v)).double()
    info = torch.finfo(dtype)
    assert bool(((o.double() - want).abs() <= want.abs() * info.eps * (1 + 2.0 ** -7) + info.smallest_normal * info.eps).all())


@pytest.mark.parametrize("score", [-1e34, -1e31, -1e9, 1e9, 1e34])
def test_one_key_has_all_the_weight_whatever_its_score(score):
    q, k = torch.zeros(2, 300, 1, 64, dtype=torch.bfloat16, device="cuda")
    q[..., 0], k[..., 0] = 8.0 * score / abs(score) * abs(score) ** 0.5, abs(score) ** 0.5
    v = randn(300, 1, 64, dtype=torch.bfloat16, seed=3)
    starts = torch.arange(301, dtype=torch.int32, device="cuda")
    o = q8.PromptAttention()(q, k, v, starts, torch.empty_like(q))
    assert torch.equal(o, v)
