"""The gated MLP block refuses bad arguments before it changes anything."""
import pytest
import torch

from fp8_implicit_gemm_gb300 import capi, q8

pytestmark = pytest.mark.gpu


def test_refused_calls_leave_the_residual_as_it_was():
    g = torch.Generator(device="cuda").manual_seed(1)
    dim, inner, rows = 256, 384, 20
    mlp = q8.MlpQ8(torch.ones(dim, dtype=torch.bfloat16, device="cuda"),
                   torch.randn(2 * inner, dim, generator=g, device="cuda"),
                   torch.randn(dim, inner, generator=g, device="cuda"), max_rows=rows)
    x, r = (torch.randn(rows, dim, generator=g, device="cuda").bfloat16() for _ in range(2))
    y = torch.zeros_like(x)
    residual = r.clone()
    for args in ((x, residual, y[:, :dim - 1]), (x, residual, y[:rows - 1]), (x, residual, y.double()),
                 (x, residual, y.cpu()), (x, residual, y.t().contiguous().t()),
                 (x, residual, y[0]), (x, residual[:rows - 1], y), (x, residual.float(), y),
                 (x[:, :dim - 1], residual[:, :dim - 1], y)):
        with pytest.raises(ValueError):
            mlp(*args)
        torch.cuda.synchronize()
        assert torch.equal(residual, r)
    mlp(x, residual, y)
    assert mlp.check() == capi.CONV3D_OK
    assert torch.equal(residual, (x.float() + r.float()).bfloat16())
    mlp.close()
