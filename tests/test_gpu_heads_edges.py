"""Heads at the ends of fp32's range whose halves are read twice, and elements behind the rotated ones beside values that
are not finite."""
import pytest
import torch

from fp8_implicit_gemm_gb300 import capi, q8
from _attention_common import heads64, randn
from test_gpu_heads import check, frequencies

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rot,dim", [(24, 64), (40, 64), (8, 8), (72, 80), (200, 256)])
@pytest.mark.parametrize("size", [2.0 ** -149, 2.0 ** -140, 1e-38, 1e-25, 1.0, 1e25, 1e37])
def test_loose_halves_of_tiny_and_huge_rows(rot, dim, size):
    """Halves that do not fill lanes: each element's partner is normed like itself, with an eps of 0 whatever the size."""
    x = (randn(5, 3, dim, seed=1).double() * size * 4).float()
    w = 1 + 0.1 * randn(dim, seed=2)
    pos = torch.arange(5, device="cuda") * 1000 + 3
    axis, freqs = torch.zeros(rot // 2, dtype=torch.int64, device="cuda"), frequencies([rot // 2])
    out = torch.empty_like(x)
    for eps in (0.0, 1.0):
        capi.heads_q8_run(q=x, q_out=out, q_weight=w, eps=eps, rotary=q8.Rotary(rot), positions=pos)
        check(out, *heads64(x, w, eps, freqs, axis, pos[None], rot))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("adjacent", [True, False])
@pytest.mark.parametrize("rot", [2, 4, 6, 8, 12, 20, 30, 32])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_elements_behind_the_rotated_ones_stay(dtype, adjacent, rot, bad):
    """Bit by bit, zeros of either sign among them, beside infinities and NaN in their own places."""
    dim = 64
    x = randn(3, 2, dim, dtype=dtype, seed=1)
    x[..., 36], x[0, :, rot] = -0.0, -0.0
    x[0, :, rot + 1], x[1, :, rot], x[2, :, 40] = bad, bad, bad
    x[2, :, rot + 1], x[2, :, rot] = -1.0, -0.0
    out = torch.empty_like(x)
    pos = torch.arange(3, device="cuda") + 5
    capi.heads_q8_run(q=x, q_out=out, rotary=q8.Rotary(rot, adjacent=adjacent), positions=pos)
    bits = torch.int16 if dtype == torch.bfloat16 else torch.int32
    a, b = out[..., rot:].contiguous(), x[..., rot:].contiguous()
    assert torch.equal(torch.isnan(a), torch.isnan(b))
    assert torch.equal(a.nan_to_num(1.0, None, None).view(bits)[~torch.isnan(b)], b.nan_to_num(1.0, None, None).view(bits)[~torch.isnan(b)])
    assert bool(torch.isfinite(out[..., :rot]).all())
