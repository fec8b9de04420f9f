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


@pytest.mark.parametrize("rows", [4, 200])
@pytest.mark.parametrize("laid_out", [True, False])
def test_layer_made_on_one_stream_and_called_on_another(rows, laid_out):
    """What a layer lays out for itself when it is made is in place for calls on every stream."""
    K = 512 if laid_out else 500
    w, sw = weights(256, K)
    w = w if laid_out else w.contiguous()
    x, sx = weights(rows, K, seed=2)
    want, y = (torch.empty(rows, 256, device="cuda") for _ in range(2))
    q8.LinearQ8(w, sw, max_rows=rows)(x, sx, want)
    torch.cuda.synchronize()
    made, called = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(made):
        torch.cuda._sleep(SLEEP)
        layer = q8.LinearQ8(w, sw, max_rows=rows)
    layer(x, sx, y, stream=called)
    assert layer.check() == capi.CONV3D_OK
    assert torch.equal(y, want)
    layer.close()


@pytest.mark.parametrize("rows", [4, 200])
def test_block_made_on_one_stream_and_called_on_another(rows):
    g = torch.Generator(device="cuda").manual_seed(3)
    w_gu = torch.randn(600, 256, generator=g, device="cuda")
    w_down = torch.randn(256, 300, generator=g, device="cuda")
    weight = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(rows, 256, generator=g, device="cuda").bfloat16()
    want, y = torch.empty_like(x), torch.empty_like(x)
    q8.MlpQ8(weight, w_gu, w_down, max_rows=rows)(x, torch.zeros_like(x), want)
    residual = torch.zeros_like(x)
    torch.cuda.synchronize()
    made, called = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(made):
        torch.cuda._sleep(SLEEP)
        mlp = q8.MlpQ8(weight, w_gu, w_down, max_rows=rows)
    mlp(x, residual, y, stream=called)
    assert mlp.check() == capi.CONV3D_OK
    assert torch.equal(y, want)
    mlp.close()
