"""What the attention block refuses is refused before the residual and the cache change."""
import pytest
import torch

from fp8_implicit_gemm_gb300 import capi, q8
from _attention_common import CODE_ARG, CODES, randn

pytestmark = pytest.mark.gpu
DIM, HEADS, KV = 128, 4, 2


def parts(head=64, codes="i8", seed=1):
    cache = q8.CacheQ8.empty(4, 16, KV, head, CODE_ARG[codes])
    w = randn((HEADS + 2 * KV) * head, DIM, seed=seed) / DIM ** 0.5
    return torch.ones(DIM, dtype=torch.bfloat16, device="cuda"), w, cache


def rows(n, head=64):
    x, residual = [randn(n, DIM, dtype=torch.bfloat16, seed=s) for s in (2, 3)]
    return x, residual, torch.arange(n, device="cuda"), torch.empty(n, HEADS, head, dtype=torch.bfloat16, device="cuda")


def whole(cache):
    return [t.view(torch.uint8).clone() for t in (cache.k_codes, cache.v_codes, cache.k_scale, cache.v_scale)]


@pytest.mark.parametrize("codes", CODES)
def test_prompts_of_256_channels(codes):
    """They are refused; the newest tokens of such heads are not."""
    weight, w, cache = parts(256, codes)
    block = q8.AttentionQ8(weight, w, HEADS, cache, q8.Rotary(256), max_rows=16)
    x, residual, at, o = rows(8, 256)
    before, kept = residual.clone(), whole(cache)
    with pytest.raises(ValueError):
        block.prompt(x, residual, torch.tensor([0, 8], dtype=torch.int32, device="cuda"), at, at, o)
    assert torch.equal(residual, before) and all(torch.equal(a, b) for a, b in zip(whole(cache), kept))
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    block.decode(x[:1], residual[:1], at[:1], at[:1], table, torch.ones(1, dtype=torch.int32, device="cuda"), o[:1])
    assert block.check() == capi.CONV3D_OK and bool(torch.isfinite(o[:1]).all())
    assert torch.equal(residual[:1], (x[:1].float() + before[:1].float()).bfloat16())


def test_parts_that_the_heads_would_refuse():
    """The block is not made of a rotary of another device, norms of another type or layout, or a cache elsewhere."""
    weight, w, cache = parts()
    norm = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    for kw in (dict(rotary=q8.Rotary(64, device="cpu")), dict(q_norm=norm.double()), dict(k_norm=norm.double()),
               dict(q_norm=norm.int(), k_norm=norm.int()), dict(q_norm=norm.cpu()), dict(k_norm=norm.cpu()),
               dict(q_norm=torch.ones(128, device="cuda")[::2])):
        with pytest.raises(ValueError):
            q8.AttentionQ8(weight, w, HEADS, cache, max_rows=16, **kw)
    with pytest.raises(ValueError):
        q8.AttentionQ8(weight.cpu(), w, HEADS, cache, max_rows=16)
    with pytest.raises(ValueError):
        q8.AttentionQ8(weight, w.cpu(), HEADS, cache, max_rows=16)


def test_missing_positions():
    weight, w, cache = parts()
    block = q8.AttentionQ8(weight, w, HEADS, cache, q8.Rotary(64), max_rows=16)
    x, residual, at, o = rows(4)
    before, kept = residual.clone(), whole(cache)
    starts, table = torch.tensor([0, 4], dtype=torch.int32, device="cuda"), torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        block.prompt(x, residual, starts, None, at, o)
    with pytest.raises(ValueError):
        block.decode(x, residual, None, at, table, torch.ones(4, dtype=torch.int32, device="cuda"), o)
    assert torch.equal(residual, before) and all(torch.equal(a, b) for a, b in zip(whole(cache), kept))
    q8.AttentionQ8(weight, w, HEADS, cache, max_rows=16).prompt(x, residual, starts, None, at, o)  # without a rotary
    assert bool(torch.isfinite(o).all())
