"""The attention block: the operators as a program uses them one after another, prompts and then token by token."""
import pytest
import torch

from fp8_implicit_gemm_gb300 import capi, q8
from _attention_common import (CODE_ARG, CODES, ROUND, attention64, check_attention, randn, values64)

pytestmark = pytest.mark.gpu
DIM, HEADS, KV, HEAD, PAGE = 320, 6, 2, 64, 16


def layer(codes, weights=torch.int8, max_rows=200, max_seqs=4, max_tokens=2, norms=True, axes=1):
    cache = q8.CacheQ8.empty(40, PAGE, KV, HEAD, CODE_ARG[codes])
    w = randn((HEADS + 2 * KV) * HEAD, DIM, seed=1) / DIM ** 0.5
    w[: HEADS * HEAD] *= 2
    rotary = q8.Rotary(HEAD, sections=None if axes == 1 else [8, 12, 12])
    n = [(1 + 0.1 * randn(HEAD, seed=s)).bfloat16() for s in (2, 3)] if norms else [None, None]
    return q8.AttentionQ8((1 + 0.1 * randn(DIM, seed=4)).bfloat16(), w, HEADS, cache, rotary, *n, max_rows=max_rows,
                          max_seqs=max_seqs, max_tokens=max_tokens, codes=weights)


@pytest.mark.parametrize("codes", CODES)
@pytest.mark.parametrize("weights", [torch.int8, torch.float8_e4m3fn])
def test_prompts_then_tokens(codes, weights):
    """Two prompts, then three steps of two tokens each: every step's output is attention over what the cache holds, in 64
    bits, and what the cache holds are the turned keys and the values of every step."""
    block, table = layer(codes, weights), torch.tensor([[5, 9, 0, 11], [7, 3, 2, 1]], dtype=torch.int32, device="cuda")
    lengths = [37, 5]
    x = randn(sum(lengths), DIM, dtype=torch.bfloat16, seed=5)
    residual = randn(sum(lengths), DIM, dtype=torch.bfloat16, seed=6)
    before = residual.clone()
    at = torch.cat([torch.arange(n, device="cuda") for n in lengths])
    seq = torch.tensor([0] * 37 + [1] * 5, device="cuda")

    def slots(seq, at):
        return table[seq, at // PAGE].long() * PAGE + at % PAGE
    starts = torch.tensor([0, 37, 42], dtype=torch.int32, device="cuda")
    o = torch.empty(42, HEADS, HEAD, dtype=torch.bfloat16, device="cuda")
    block.prompt(x, residual, starts, at, slots(seq, at), o)
    assert block.check() == capi.CONV3D_OK
    assert torch.equal(residual, (x.float() + before.float()).bfloat16())
    q, k, v = [t.clone() for t in block._qkv[:42].split([HEADS, KV, KV], dim=1)]
    for a, e in ((0, 37), (37, 42)):
        limits = torch.arange(1, e - a + 1, device="cuda")
        want, size, worst = attention64(q[a:e], k[a:e], v[a:e], limits, HEAD ** -0.5)
        check_attention(o[a:e], want, size, worst, ROUND[o.dtype], e - a)
    # the cache holds codes of the keys (not rounded to 16 bits before) and of the values
    kb, vb = torch.empty(2, 42, KV, HEAD, dtype=torch.bfloat16, device="cuda")
    block.cache.read(slots(seq, at), kb, vb)
    steps = {"i4": 15.0, "i8": 254.0, "e4m3": 2 * 448.0}[codes]
    for got, t in ((kb, k), (vb, v)):
        width = t.float().abs().amax(-1, keepdim=True) * 2
        # half a code's step (an e4m3 code: 2^-4 of it), and both roundings to 16 bits
        bound = width / steps / 2 * 1.01 + t.float().abs() * (2.0 ** -4 if codes == "e4m3" else 0) + width * 2.0 ** -8
        assert bool(((got.float() - t.float()).abs() <= bound).all())
    for step in range(3):
        new = torch.tensor([[37 + 2 * step, 38 + 2 * step], [5 + 2 * step, 6 + 2 * step]], device="cuda").flatten()
        which = torch.tensor([0, 0, 1, 1], device="cuda")
        x, residual = randn(4, DIM, dtype=torch.bfloat16, seed=10 + step), torch.zeros(4, DIM, dtype=torch.bfloat16, device="cuda")
        o = torch.empty(4, HEADS, HEAD, dtype=torch.bfloat16, device="cuda")
        n = torch.tensor([39 + 2 * step, 7 + 2 * step], dtype=torch.int32, device="cuda")
        block.decode(x, residual, new, slots(which, new), table, n, o)
        assert block.check() == capi.CONV3D_OK
        k64, v64 = values64(block.cache, "k", codes), values64(block.cache, "v", codes)
        for b in range(2):
            k, v = [t[table[b].long()].transpose(1, 2).flatten(0, 1)[:int(n[b])] for t in (k64, v64)]
            limits = int(n[b]) - 1 + torch.arange(2, device="cuda")
            rows = slice(2 * b, 2 * b + 2)
            want, size, worst = attention64(block._qkv[rows, :HEADS], k, v, limits, HEAD ** -0.5)
            check_attention(o[rows], want, size, worst, 2.0 ** -11, int(n[b]))
    block.close()


def test_the_block_is_its_calls():
    """Bit by bit what the library's calls give one after another; with several axes of positions, without norms."""
    block = layer("i8", norms=False, axes=3)
    x, residual = randn(60, DIM, dtype=torch.bfloat16, seed=5), randn(60, DIM, dtype=torch.bfloat16, seed=6)
    r, pos = residual.clone(), torch.randint(0, 50, (3, 60), device="cuda")
    slots, starts = torch.arange(60, device="cuda") * 3, torch.tensor([0, 60], dtype=torch.int32, device="cuda")
    o = torch.empty(60, HEADS, HEAD, dtype=torch.bfloat16, device="cuda")
    block.prompt(x, residual, starts, pos, slots, o)
    a, scale = q8.empty_codes(60, DIM), torch.empty(60, device="cuda")
    capi.rmsnorm_q8_run(x, block.norm_weight, a, scale, 1e-6, residual=r, residual_out=r)
    qkv = block.qkv(a, scale, torch.empty(60, (HEADS + 2 * KV) * HEAD, dtype=torch.bfloat16, device="cuda")).view(60, -1, HEAD)
    q, k, v = qkv.split([HEADS, KV, KV], dim=1)
    cache = q8.CacheQ8.empty(40, PAGE, KV, HEAD)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    capi.heads_q8_run(q=q, q_out=qo, k=k, k_out=ko, v=v, rotary=block.rotary, positions=pos, cache=cache, slots=slots)
    want = q8.PromptAttention()(qo, ko, v, starts, torch.empty_like(o))
    assert torch.equal(residual, r) and torch.equal(o, want)
    assert torch.equal(cache.k_codes, block.cache.k_codes) and torch.equal(cache.v_scale, block.cache.v_scale)


def test_made_on_one_stream_captured_and_replayed_on_another():
    made, called = torch.cuda.Stream(), torch.cuda.Stream()
    x = randn(2, DIM, dtype=torch.bfloat16, seed=5)
    residual, o = torch.zeros_like(x), torch.empty(2, HEADS, HEAD, dtype=torch.bfloat16, device="cuda")
    pos, slots = torch.tensor([3, 3], device="cuda"), torch.tensor([3, 35], device="cuda")
    table, n = torch.tensor([[0], [2]], dtype=torch.int32, device="cuda"), torch.tensor([4, 4], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(made):
        torch.cuda._sleep(50_000_000)
        block = layer("i4")
    with torch.cuda.stream(called):
        block.decode(x, residual, pos, slots, table, n, o)
        want = o.clone()
        graph = torch.cuda.CUDAGraph()
        residual.zero_()
        called.synchronize()
        with torch.cuda.graph(graph, stream=called):
            residual.zero_()
            block.decode(x, residual, pos, slots, table, n, o)
    o.zero_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert block.check() == capi.CONV3D_OK and torch.equal(o, want) and bool(torch.isfinite(o).all())


def test_refusals_leave_the_residual():
    block = layer("i8", max_rows=8)
    x, residual = randn(4, DIM, dtype=torch.bfloat16, seed=5), randn(4, DIM, dtype=torch.bfloat16, seed=6)
    before, at = residual.clone(), torch.arange(4, device="cuda")
    starts = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    table, n = torch.zeros(4, 1, dtype=torch.int32, device="cuda"), torch.ones(4, dtype=torch.int32, device="cuda")
    o = torch.empty(4, HEADS, HEAD, dtype=torch.bfloat16, device="cuda")
    for args in ((starts, at, at, o[:3]), (starts, at, at, o.float()), (starts, at[:3], at, o), (starts, at, at.int(), o),
                 (starts.long(), at, at, o), (starts, at.int(), at, o)):
        with pytest.raises(ValueError):
            block.prompt(x, residual, *args)
    for args in ((at, at, table.long(), n, o), (at, at, table, n[:3], o), (at, at, table[:3], n[:3], o), (at, at, table, n, o[:, :3])):
        with pytest.raises(ValueError):
            block.decode(x, residual, *args)
    with pytest.raises(ValueError):
        block.prompt(torch.cat([x] * 3), torch.cat([residual] * 3), starts, torch.arange(12, device="cuda"),
                     torch.arange(12, device="cuda"), torch.cat([o] * 3))
    assert torch.equal(residual, before)
    with pytest.raises(ValueError):
        q8.AttentionQ8(block.norm_weight, randn(64, DIM), HEADS, block.cache)


def test_demo_runs():
    q8._demo_attention()


def test_what_attention_would_refuse_leaves_the_residual():
    block = layer("i8", max_rows=16)
    x, residual = randn(8, DIM, dtype=torch.bfloat16, seed=5), randn(8, DIM, dtype=torch.bfloat16, seed=6)
    before, at = residual.clone(), torch.arange(8, device="cuda")
    starts = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    o = torch.empty(8, HEADS, HEAD, dtype=torch.bfloat16, device="cuda")
    spare = torch.empty(8 * HEADS * HEAD + 8, dtype=torch.bfloat16, device="cuda")
    outputs = (spare[1:1 + o.numel()].view(o.shape), spare.as_strided(o.shape, (HEADS * HEAD - 1, HEAD, 1)),
               o[:1].expand(o.shape), o[:, :1].expand(o.shape), spare.as_strided(o.shape, (HEAD, HEAD, 1)))
    for bad in ((starts[:0], at, at, o), (starts[None], at, at, o), *((starts, at, at, out) for out in outputs),
                (starts, torch.arange(16, device="cuda")[::2], at, o)):
        with pytest.raises(ValueError):
            block.prompt(x, residual, *bad)

    def table(seqs, width=1):
        return torch.zeros(seqs, width, dtype=torch.int32, device="cuda"), torch.ones(seqs, dtype=torch.int32, device="cuda")
    for t, n in (table(8), table(2), table(1), table(4, 0)):  # too many sequences, too many tokens, twice, no pages
        with pytest.raises(ValueError):
            block.decode(x, residual, at, at, t, n, o)
    with pytest.raises(ValueError):
        block.decode(x, residual, at, at, table(1, 2)[0].expand(4, 2), table(4)[1], o)
    assert torch.equal(residual, before) and block.check() == capi.CONV3D_OK
    with pytest.raises(ValueError):
        q8.AttentionQ8(block.norm_weight.float(), randn((HEADS + 2 * KV) * HEAD, DIM), HEADS, block.cache)


def test_outputs_with_heads_ahead_of_tokens():
    """An output in the order [heads, tokens], and positions that all axes share."""
    x, residual = randn(8, DIM, dtype=torch.bfloat16, seed=5), randn(8, DIM, dtype=torch.bfloat16, seed=6)
    at, starts = torch.arange(8, device="cuda"), torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    o = torch.empty(8, HEADS, HEAD, dtype=torch.bfloat16, device="cuda")
    other = torch.empty(HEADS, 8, HEAD, dtype=torch.bfloat16, device="cuda")
    layer("i8", axes=3).prompt(x, residual.clone(), starts, at.expand(3, 8).contiguous(), at, o)
    layer("i8", axes=3).prompt(x, residual.clone(), starts, at.expand(3, 8), at, other.transpose(0, 1))
    assert torch.equal(o, other.transpose(0, 1)) and bool(torch.isfinite(o).all())
