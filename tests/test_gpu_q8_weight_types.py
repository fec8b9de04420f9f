"""A norm's weight of every type beside rows of every type, in every kernel."""
import pytest
import torch

from fp8_implicit_gemm_gb300 import capi
from _q8_common import U, VALUE_TYPES, check_codes, norm64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols,pitch,offset", [
    (200, 208, 0), (4096, 4096, 0), (9000, 9008, 0), (12300, 12304, 0), (20000, 20000, 0),
    (32768, 32768, 0), (1001, 1017, 1), (4098, 4102, 2), (12501, 12517, 1), (12502, 12504, 2)])
@pytest.mark.parametrize("weight_dtype", VALUE_TYPES)
@pytest.mark.parametrize("dtype", VALUE_TYPES)
def test_weight_types(dtype, weight_dtype, cols, pitch, offset):
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.empty(5, pitch, dtype=dtype, device="cuda")[:, offset:offset + cols]
    x.copy_(torch.randn(5, cols, generator=g, device="cuda"))
    for at in (0, offset):  # the weight's own alignment
        weight = torch.empty(cols + 8, dtype=weight_dtype, device="cuda")[at:at + cols]
        weight.copy_(1 + 0.1 * torch.randn(cols, generator=g, device="cuda"))
        q, scale = torch.empty(5, cols, dtype=torch.int8, device="cuda"), torch.empty(5, device="cuda")
        capi.rmsnorm_q8_run(x, weight, q, scale, 1e-6)
        check_codes(q, scale, norm64(x, weight, 1e-6)[1], 16 * U, 2.0 ** -17)
