"""Plans and layers with work on more than one stream."""
import pytest
import torch

from fp8_implicit_gemm_gb300 import capi, q8

pytestmark = pytest.mark.gpu
SLEEP = 100_000_000  # cycles: some 50 ms


def weights(N, K, code_dtype=torch.int8, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return q8.quantise_rows(torch.randn(N, K, generator=g, device="cuda"), code_dtype)


@pytest.mark.parametrize("rows", [4, 200])
def test_destroy_waits_for_the_device(rows):
    """Also where the plan holds no device memory: what its runs read may be freed once it returns."""
    w, sw = weights(256, 512)
    x, sx = weights(rows, 512, seed=2)
    y = torch.empty(rows, 256, device="cuda")
    plan = capi.linear_q8_plan(rows, 256, 512, capi.Q8_INT8, 0)
    assert (capi.linear_q8_workspace_size(plan) == 0) == (rows == 4)
    capi.linear_q8_run(plan, x, sx, w, sw, y)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(SLEEP)
    capi.linear_q8_run(plan, x, sx, w, sw, y, stream=s)
    assert not s.query()
    capi.linear_q8_destroy(plan)
    assert s.query()
