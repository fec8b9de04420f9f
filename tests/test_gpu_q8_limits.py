"""The row operators' shared memory: rows around the default limit of a block, each as the first wide
call of a process."""
import os
import subprocess
import sys

import pytest

REPO_ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu

# A process of its own: a kernel's shared-memory limit outlasts the call that raised it.
FIRST_CALL = """
import sys
import torch
sys.path[:0] = [{root!r}, {tests!r}]
from fp8_implicit_gemm_gb300 import capi
from _q8_common import U, act64, check_codes, norm64
cols, pitch, dtype = {cols}, {pitch}, torch.{dtype}
g = torch.Generator(device="cuda").manual_seed(cols)
x = torch.empty(3, pitch, dtype=dtype, device="cuda")[:, :cols]
up = torch.empty(3, pitch, dtype=dtype, device="cuda")[:, :cols]
x.copy_(torch.randn(3, cols, generator=g, device="cuda"))
up.copy_(torch.randn(3, cols, generator=g, device="cuda"))
weight = torch.ones(cols, dtype=dtype, device="cuda")
q = torch.empty(3, cols, dtype=torch.int8, device="cuda")
scale = torch.empty(3, device="cuda")
if {norm}:
    capi.rmsnorm_q8_run(x, weight, q, scale, 1e-6)
    check_codes(q, scale, norm64(x, weight, 1e-6)[1], 16 * U, 2.0 ** -17)
else:
    capi.silu_mul_q8_run(x, up, q, scale)
    err = 2 * (float(x.abs().max()) + 4) * U + 16 * U
    check_codes(q, scale, act64(x, up), 2 * err, err)
"""


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("cols", [12160, 12161, 12287, 12288])
@pytest.mark.parametrize("dtype,off_grid", [("float32", 0), ("bfloat16", 1), ("float16", 2)])
def test_first_wide_call_of_a_process(dtype, off_grid, cols, norm):
    """The values of such a row and the reduction's 512 bytes together pass 48 KB from 12161 columns
    on, the values alone from 12289."""
    pitch = -(-cols // 16) * 16 + off_grid
    script = FIRST_CALL.format(root=REPO_ROOT, tests=os.path.join(REPO_ROOT, "tests"), cols=cols,
                               pitch=pitch, dtype=dtype, norm=norm)
    r = subprocess.run([sys.executable, "-c", script], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
