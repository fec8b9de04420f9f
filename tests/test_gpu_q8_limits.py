"""The row operators' shared memory: rows around the default limit of a block, each as the first wide
call of a process, and two host threads with rows of two widths."""
import ctypes
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


# Two host threads that do nothing but call: a thread of the interpreter holds its lock between calls.
TWO_CALLERS = r"""
#include <thread>
extern "C" void two_callers(int (*run)(const void*), const void* a, const void* b, int rounds,
                            int* refused) {
  auto calls = [=](const void* args, int* n) {
    for (int i = 0; i < rounds; ++i) *n += run(args) != 0;
  };
  std::thread t(calls, a, refused), u(calls, b, refused + 1);
  t.join();
  u.join();
}
"""


def test_two_host_threads_with_rows_of_two_widths(tmp_path):
    """Calls of two threads, each on a stream of its own, whose rows need different amounts of shared
    memory of one kernel: none is refused, and each gives what it gives alone."""
    import torch

    from fp8_implicit_gemm_gb300 import capi
    src, so = tmp_path / "callers.cpp", tmp_path / "callers.so"
    src.write_text(TWO_CALLERS)
    subprocess.run(["g++", "-shared", "-fPIC", "-pthread", "-O1", str(src), "-o", str(so)], check=True)
    lib = capi.load()
    args, data = [], []
    for cols in (12504, 32000):
        g = torch.Generator(device="cuda").manual_seed(cols)
        x = torch.randn(2, cols, generator=g, device="cuda")
        weight = torch.ones(cols, device="cuda")
        first = torch.empty(2, cols, dtype=torch.int8, device="cuda"), torch.empty(2, device="cuda")
        again = torch.empty_like(first[0]), torch.empty_like(first[1])
        capi.rmsnorm_q8_run(x, weight, *first, 1e-6)
        stream = torch.cuda.Stream()
        args.append(capi._RMSNORM_ARGS.pack(
            x.data_ptr(), 0, weight.data_ptr(), 0, again[0].data_ptr(), again[1].data_ptr(), cols, 0,
            0, cols, 2, cols, stream.cuda_stream, capi.Q8_F32, capi.Q8_F32, capi.Q8_INT8, 0, 1e-6, 0))
        data.append((x, weight, first, again, stream))
    torch.cuda.synchronize()
    refused = (ctypes.c_int * 2)()
    run = ctypes.cast(lib.rmsnorm_q8_run, ctypes.c_void_p)
    ctypes.CDLL(str(so)).two_callers(run, ctypes.c_char_p(args[0]), ctypes.c_char_p(args[1]), 20000,
                                     refused)
    torch.cuda.synchronize()
    assert list(refused) == [0, 0]
    for _, _, first, again, _ in data:
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
