"""Scales of scores next to 0, and 0, beside scores of any size."""
import pytest
import torch

from fp8_implicit_gemm_gb300 import capi, q8
from _attention_common import ROUND, attention64, check_attention, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("size", [1.0, 1e9, 1e17])
def test_a_scale_of_0_is_the_mean(size, causal):
    """Whatever the scores before it (up to 1e36 here), and infinite ones of keys that are not seen."""
    n, dim = 300, 64
    q, k = [(size * randn(n, 2, dim, seed=s)).bfloat16() for s in (1, 2)]
    v = randn(n, 2, dim, dtype=torch.bfloat16, seed=3)
    starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    attend = q8.PromptAttention(scale=0.0)
    o = attend(q, k, v, starts, torch.empty_like(q), causal=causal)
    assert attend.check() == capi.CONV3D_OK
    limits = torch.arange(1, n + 1, device="cuda") if causal else torch.full((n,), n, device="cuda")
    want, sizes, _ = attention64(q, k, v, limits, 0.0)
    check_attention(o, want, sizes, 0.0, ROUND[o.dtype], n)


@pytest.mark.parametrize("scale,size", [(1e-33, 1e16), (-1e-33, 1e16), (2e-38, 3e18), (1e-40, 3e18), (1e-31, 1e3)])
def test_small_scales_are_not_replaced(scale, size):
    n, dim = 200, 64
    q, k = [(size * randn(n, 1, dim, seed=s)).bfloat16() for s in (1, 2)]
    v = randn(n, 1, dim, dtype=torch.bfloat16, seed=3)
    starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    o = q8.PromptAttention(scale=scale)(q, k, v, starts, torch.empty_like(q), causal=False)
    # scores are fp32: of the 40000 products of values of 3e18 one is -3.48e38, past its range, and its row is left out
    inside = (q.double()[:, 0] @ k.double()[:, 0].t()).abs().amax(dim=1) <= torch.finfo(torch.float32).max
    assert int(inside.sum()) >= n - 1
    o, q = o[inside], q[inside]
    want, sizes, worst = attention64(q, k, v, torch.full((o.shape[0],), n, device="cuda"), scale)
    # a scale below fp32's normal numbers is rounded to a multiple of 2^-149 there, and its product with log2(e) again
    worst += float((q.double()[:, 0] @ k.double()[:, 0].t()).abs().max()) * 2.0 ** -148
    check_attention(o, want, sizes, worst, ROUND[o.dtype], n)


def test_the_largest_scales():
    """Equal scores have equal weights, and 0 is one of them."""
    n, dim = 150, 64
    q = torch.zeros(n, 1, dim, dtype=torch.bfloat16, device="cuda")
    k, v = randn(n, 1, dim, dtype=torch.bfloat16, seed=2), randn(n, 1, dim, dtype=torch.bfloat16, seed=3)
    starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    for scale in (3.4e38, -3.4e38, 1e38):
        o = q8.PromptAttention(scale=scale)(q, k, v, starts, torch.empty_like(q), causal=False)
        want, sizes, _ = attention64(q, k, v, torch.full((n,), n, device="cuda"), 0.0)
        check_attention(o, want, sizes, 0.0, ROUND[o.dtype], n)
