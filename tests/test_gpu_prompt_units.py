"""Blocks of the prompt kernel that pass through units of one to several tiles of keys, or none, in any order: a unit's first
copy falls on every slot of the ring, and copies of several units are under way together."""
import pytest
import torch

from fp8_implicit_gemm_gb300 import capi, q8
from _attention_common import ROUND, attention64, check_attention, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_units_of_all_lengths(dtype, dim, causal):
    """300 sequences x 4 heads of 1 to 300 queries over 0 to 900 keys: some four units a block, of 0 to 8 tiles, with tiles of
    rows that see nothing in front of ones that do."""
    g = torch.Generator().manual_seed(dim + causal)
    lengths = torch.randint(1, 301, (300,), generator=g)
    keys = torch.where(torch.rand(300, generator=g) < 0.5, torch.randint(0, 300, (300,), generator=g),
                       torch.randint(0, 901, (300,), generator=g))
    starts, key_starts = [torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)]).int().cuda() for n in (lengths, keys)]
    q = randn(int(starts[-1]), 4, dim, dtype=dtype, seed=1)
    k, v = [randn(int(key_starts[-1]), 2, dim, dtype=dtype, seed=s) for s in (2, 3)]
    attend = q8.PromptAttention()
    o = attend(q, k, v, starts, torch.full_like(q, 7.0), causal=causal, key_starts=key_starts)
    assert attend.check() == capi.CONV3D_OK
    for _ in range(10):
        assert torch.equal(attend(q, k, v, starts, torch.full_like(q, 7.0), causal=causal, key_starts=key_starts), o)
    assert attend.check() == capi.CONV3D_OK
    a = c = 0
    for n, m in zip(lengths.tolist(), keys.tolist()):
        limits = torch.full((n,), m, device="cuda")
        if causal:
            limits = (torch.arange(1, n + 1, device="cuda") + m - n).clamp(min=0)
        want, size, worst = attention64(q[a:a + n], k[c:c + m], v[c:c + m], limits, dim ** -0.5)
        check_attention(o[a:a + n], want, size, worst, ROUND[dtype], m, f"{n} queries over {m} keys")
        a, c = a + n, c + m
