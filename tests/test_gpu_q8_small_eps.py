"""The norm with an eps of 0 or next to it, on rows whose squares underflow fp32."""
import pytest
import torch

from fp8_implicit_gemm_gb300 import capi
from _q8_common import CODE_TYPES, U, check_codes, check_values, norm64

pytestmark = pytest.mark.gpu
CODE_ERR, SCALE_ERR = 16 * U, 2.0 ** -17
# each row's size; 1e-19 to 1e-22 have subnormal squares, from 1e-23 on squares are 0
SIZES = [1.0, 1e-8, 1e-14, 1e-16, 1e-18, 1e-19, 1e-20, 1e-22, 1e-25, 1e-30, 1e-36, 1e15]


def rows_of_sizes(cols, pitch, offset, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.zeros(len(SIZES) + 3, pitch, dtype=dtype, device="cuda")[:, offset:offset + cols]
    size = torch.tensor(SIZES, device="cuda")[:, None]
    x[:len(SIZES)] = (torch.randn(len(SIZES), cols, generator=g, device="cuda") * size).to(dtype)
    # a row of zeros; one small value behind zeros; small values before an ordinary one
    x[-2, cols - 1] = 1e-25
    x[-1] = (torch.randn(cols, generator=g, device="cuda") * 1e-25).to(dtype)
    x[-1, cols - 1] = 2.0
    return x


@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-37, 1e-36])
@pytest.mark.parametrize("cols,pitch,offset", [
    (1, 16, 0), (8, 8, 0), (200, 208, 0), (4096, 4096, 0), (16384, 16384, 0), (32768, 32768, 0),
    (1001, 1017, 1), (4098, 4102, 2), (12501, 12517, 1), (12502, 12504, 2)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_small_rows(dtype, cols, pitch, offset, eps):
    """Every kernel, with and without a residual, which is updated in place."""
    eps = torch.tensor(eps, dtype=torch.float32).item()  # as the call takes it: 1e-45 is 1.4e-45
    x = rows_of_sizes(cols, pitch, offset, dtype, cols)
    r = rows_of_sizes(cols, pitch, offset, dtype, cols + 1)
    weight = (1 + 0.1 * torch.randn(cols, device="cuda")).to(dtype)
    for code_dtype in CODE_TYPES:
        for residual in (None, r.clone(memory_format=torch.contiguous_format), r):
            q = torch.empty(x.shape, dtype=code_dtype, device="cuda")
            scale = torch.empty(x.shape[0], device="cuda")
            h, y = norm64(x, weight, eps, residual)
            y = torch.where((h == 0).all(dim=1, keepdim=True), 0.0, y)  # 0 / sqrt(0), if eps is 0
            before = None if residual is None else residual.clone()
            capi.rmsnorm_q8_run(x, weight, q, scale, eps, residual=residual, residual_out=residual)
            check_codes(q, scale, y, CODE_ERR, SCALE_ERR, f"{cols} {code_dtype}")
            assert float(scale[len(SIZES)]) == 1.0
            if residual is not None:
                check_values(residual, h, h.abs() * U)
                residual.copy_(before)


def test_subnormal_rows():
    """Rows of subnormal values and a weight of ones: y keeps all bits that x has."""
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(4, 4096, generator=g, device="cuda")
    x *= torch.tensor([1e-38, 1e-40, 1e-42, 1e-44], device="cuda")[:, None]
    weight = torch.ones(4096, device="cuda")
    for code_dtype in CODE_TYPES:
        q, scale = torch.empty(4, 4096, dtype=code_dtype, device="cuda"), torch.empty(4, device="cuda")
        capi.rmsnorm_q8_run(x, weight, q, scale, 0.0)
        check_codes(q, scale, norm64(x, weight, 0.0)[1], CODE_ERR, SCALE_ERR)


def test_many_rows_and_a_graph():
    """More rows than warps are resident, in stream order behind the work that makes them."""
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(50001, 136, generator=g, device="cuda")
    x[::7] *= 1e-24
    small = torch.empty_like(x)
    weight = torch.ones(136, device="cuda")
    q, scale = torch.empty(50001, 136, dtype=torch.int8, device="cuda"), torch.empty(50001, device="cuda")
    small.copy_(x)
    capi.rmsnorm_q8_run(small, weight, q, scale, 0.0)
    torch.cuda.synchronize()
    check_codes(q, scale, norm64(x, weight, 0.0)[1], CODE_ERR, SCALE_ERR)
    want = q.clone(), scale.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        small.copy_(x)
        capi.rmsnorm_q8_run(small, weight, q, scale, 0.0)
    q.zero_()
    scale.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(q, want[0]) and torch.equal(scale, want[1])
