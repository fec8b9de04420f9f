"""Waits that run out: the attention kernels give up, say so, and leave everything usable."""
import pytest
import torch

from fp8_implicit_gemm_gb300 import capi, q8
from _attention_common import CODE_ARG, fill_cache, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("codes", ["i4", "i8"])
@pytest.mark.parametrize("lengths", [[2000], [64, 500, 33] * 4, [40] * 300])
def test_cache_attention_gives_up(codes, lengths):
    seqs, heads, kv, dim = len(lengths), 8, 2, 128
    width = -(-max(lengths) // 16)
    cache = q8.CacheQ8.empty(seqs * width, 16, kv, dim, CODE_ARG[codes])
    fill_cache(cache, codes, 1)
    table = torch.arange(seqs * width, dtype=torch.int32, device="cuda").view(seqs, width)
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    q = randn(seqs, heads, dim, dtype=torch.bfloat16, seed=2)
    good = q8.CacheAttention(cache, heads, max_seqs=seqs)
    want = good(q, table, n, torch.empty_like(q)).clone()
    plan = capi.attn_q8_plan(seqs, 1, heads, kv, dim, cache.code_type, wait_timeout_ms=20, debug_flags=1)
    guard = torch.full((seqs + 2, heads, dim), 7.0, dtype=q.dtype, device="cuda")
    for _ in range(2):
        capi.attn_q8_run(plan, q, cache, table, n, guard[1:-1], dim ** -0.5)
        assert capi.attn_q8_check(plan) == capi.CONV3D_EDEVICE
        assert capi.attn_q8_check(plan) == capi.CONV3D_OK
    assert bool((guard[0] == 7.0).all() and (guard[-1] == 7.0).all())
    assert bool(torch.isnan(guard[1:-1]).any())
    capi.attn_q8_destroy(plan)
    assert torch.equal(good(q, table, n, torch.empty_like(q)), want) and good.check() == capi.CONV3D_OK


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rows", [100, 3000])
def test_prompt_attention_gives_up(dim, rows):
    q, k, v = [randn(rows, 2, dim, dtype=torch.bfloat16, seed=s) for s in range(3)]
    starts = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    good = q8.PromptAttention()
    want = good(q, k, v, starts, torch.empty_like(q)).clone()
    plan = capi.attn_prompt_plan(0, wait_timeout_ms=20, debug_flags=1)
    guard = torch.full((rows + 2, 2, dim), 7.0, dtype=q.dtype, device="cuda")
    for _ in range(2):
        capi.attn_prompt_run(plan, q, k, v, starts, guard[1:-1], dim ** -0.5)
        assert capi.attn_prompt_check(plan) == capi.CONV3D_EDEVICE
        assert capi.attn_prompt_check(plan) == capi.CONV3D_OK
    assert bool((guard[0] == 7.0).all() and (guard[-1] == 7.0).all())
    assert bool((guard[1:-1, 0] == 7.0).all(1).any())  # what the first block would have written
    capi.attn_prompt_destroy(plan)
    assert torch.equal(good(q, k, v, starts, torch.empty_like(q)), want) and good.check() == capi.CONV3D_OK


def test_thousands_of_short_prompts():
    """There are more blocks than units: those behind the last unit are passed over."""
    lengths = [1, 0, 2, 0, 0, 3] * 1500
    starts = torch.tensor([0] + lengths, device="cuda").cumsum(0).int()
    rows = sum(lengths)
    q, k, v = [randn(rows, 4, 64, dtype=torch.float16, seed=s) for s in range(3)]
    attend = q8.PromptAttention()
    o = attend(q, k, v, starts, torch.full_like(q, 7.0))
    assert attend.check() == capi.CONV3D_OK
    seq = torch.repeat_interleave(torch.arange(len(lengths), device="cuda"), torch.tensor(lengths, device="cuda"))
    first = starts[seq].long()
    at = torch.arange(rows, device="cuda")
    keys = (first[:, None] + torch.arange(3, device="cuda")).clamp(max=rows - 1)
    seen = first[:, None] + torch.arange(3, device="cuda") <= at[:, None]
    x = torch.einsum("rhd,rkhd->rhk", q.double(), k.double()[keys]) / 8.0
    p = torch.softmax(x.masked_fill(~seen[:, None], -torch.inf), dim=-1)
    want = torch.einsum("rhk,rkhd->rhd", p, v.double()[keys])
    # at most 3 keys: scores err by 2^-14, weights by 2^-11, the output by 2^-11 of values that are below 6
    assert float((o.double() - want).abs().max()) <= 6 * (2.0 ** -11 + 2.0 ** -11 + 2.0 ** -12)


def test_negative_timeouts_are_refused():
    for make in (lambda: capi.attn_q8_plan(1, 1, 8, 2, 128, capi.Q8_INT8, wait_timeout_ms=-1),
                 lambda: capi.attn_prompt_plan(0, wait_timeout_ms=-1)):
        with pytest.raises(capi.Conv3dFp8Error):
            make()
