"""The host side of the 8-bit products' planning, as far as it goes without a GPU."""
import ctypes
import os
import subprocess

import pytest
import torch

from fp8_implicit_gemm_gb300 import build, capi, q8

# Asks for the tiling of M x N x K, with room for 76 clusters of each size.
DECIDE = r"""
#include <cstdio>
#include <cstdlib>
#include "q8_internal.h"
int main(int argc, char** argv) {
  c3d::LinearParams p{};
  c3d::TcLimits lim{};
  p.M = atoi(argv[1]);
  p.N = atoi(argv[2]);
  p.K = atoi(argv[3]);
  lim.block_t = atoi(argv[5]);
  lim.splits = atoi(argv[6]);
  for (int& c : lim.clusters) c = 76;
  c3d::linear_tc_decide(p, atoi(argv[4]), lim);
  printf("%d %d %d %d\n", p.block_t, p.splits, p.stages, p.x_slots);
}
"""
INT8, E4M3 = 1, 2


@pytest.fixture(scope="module")
def decide(tmp_path_factory):
    build.build()
    d = tmp_path_factory.mktemp("decide")
    src, exe = d / "decide.cpp", d / "decide"
    src.write_text(DECIDE)
    cuda = os.path.dirname(os.path.dirname(build._nvcc()))
    subprocess.run(["g++", "-std=c++17", "-I", build.CSRC, "-I", build.INCLUDE, "-I",
                    os.path.join(cuda, "include"), str(src), build.LIB_PATH, "-o", str(exe),
                    f"-Wl,-rpath,{os.path.dirname(build.LIB_PATH)}"], check=True)

    def run(*args):
        r = subprocess.run([str(exe)] + [str(a) for a in args], capture_output=True, text=True)
        assert r.returncode == 0, (args, r.returncode, r.stderr)
        return [int(v) for v in r.stdout.split()]
    return run


@pytest.mark.parametrize("code_type", [INT8, E4M3])
@pytest.mark.parametrize("M,N,K,block_t,splits", [
    (40, 64, 200, 96, 0),          # a tile of more tokens than there are
    (40, 64, 200, 0, 4),           # more slices than K has blocks
    (4096, 4096, 4096, 128, 4)])   # more tiles than clusters of eight are held
def test_options_that_leave_no_tiling_end_in_none(decide, code_type, M, N, K, block_t, splits):
    """The run then reports it; the choice itself must not divide by what it has not found."""
    assert decide(M, N, K, code_type, block_t, splits)[0] == 0


@pytest.mark.parametrize("block_t", [224, 256])
def test_int8_has_no_tile_of_more_than_192_tokens(decide, block_t):
    assert decide(1000, 64, 200, INT8, block_t, 0)[0] == 0
    assert decide(1000, 64, 200, E4M3, block_t, 0)[0] == block_t


@pytest.mark.parametrize("code_type", [INT8, E4M3])
def test_free_choice_always_finds_a_tiling(decide, code_type):
    for M in (1, 33, 256, 5000):
        for N in (1, 300, 20000):
            for K in (1, 129, 1000, 30000):
                block_t, splits, stages, x_slots = decide(M, N, K, code_type, 0, 0)
                assert block_t % 32 == 0 and 32 <= block_t < M + 32
                assert 1 <= splits <= 4 and stages >= 2
                assert x_slots >= 2 if code_type == INT8 else x_slots == 0


@pytest.mark.parametrize("block_t", [224, 256])
def test_plan_refuses_int8_tiles_of_more_than_192_tokens(block_t):
    h, o = ctypes.c_void_p(1), capi.LinearOptions(block_t=block_t)
    st = capi.load().linear_q8_plan_ex(ctypes.byref(h), 1000, 64, 200, INT8, 0, ctypes.byref(o))
    assert st == capi.CONV3D_EINVAL and h.value is None


def test_block_check_reports_and_clears_both_products():
    """A status is reported once: what the second product has to report is not left for a later
    check when the first has something to report too."""
    class Layer:
        def __init__(self, *statuses):
            self.statuses = list(statuses)

        def check(self):
            return self.statuses.pop(0) if self.statuses else capi.CONV3D_OK

    mlp = q8.MlpQ8.__new__(q8.MlpQ8)
    for first, second in ((capi.CONV3D_EDEVICE, capi.CONV3D_EDEVICE),
                          (capi.CONV3D_EDEVICE, capi.CONV3D_OK),
                          (capi.CONV3D_OK, capi.CONV3D_EDEVICE)):
        mlp.gate_up, mlp.down = Layer(first), Layer(second)
        assert mlp.check() == capi.CONV3D_EDEVICE
        assert mlp.check() == capi.CONV3D_OK
    mlp.gate_up, mlp.down = Layer(), Layer(capi.CONV3D_ECUDA)
    assert mlp.check() == capi.CONV3D_ECUDA


@pytest.mark.parametrize("dtype", [torch.int8, torch.float8_e4m3fn])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_rows_that_are_not_finite_have_the_scale_nan_and_codes_0(dtype, bad):
    """As the norm and the activation mark them, so that a product of such a row is NaN."""
    v = torch.randn(4, 70, generator=torch.Generator().manual_seed(1))
    q0, s0 = q8.quantise_rows(v, dtype)
    v[2, 33] = bad
    q, s = q8.quantise_rows(v, dtype)
    keep = [0, 1, 3]
    assert torch.equal(s[keep], s0[keep])
    assert torch.equal(q[keep].view(torch.uint8), q0[keep].view(torch.uint8))
    assert bool(torch.isnan(s[2])) and float(q[2].float().abs().max()) == 0.0


@pytest.mark.parametrize("dtype,top", [(torch.int8, 127.0), (torch.float8_e4m3fn, 448.0)])
@pytest.mark.parametrize("size", [2.0 ** -126, 2.0 ** -135, 2.0 ** -142, 2.0 ** -149])
def test_rows_whose_scale_is_subnormal_keep_their_codes(dtype, top, size):
    """amax / top is then rounded coarsely, or to 0: the codes are those of the exact quotient all the
    same. The values are powers of two, which every type holds, so that quotient is one of
    top * 2^-k; the nearest code to it is within half a step (int8: 0.5, e4m3: 2^-4 of it)."""
    v = torch.tensor([[1.0, -0.5, 0.25, 0.0]]) * size
    q, _ = q8.quantise_rows(v, dtype)
    t = v.double() / (size / top)
    step = 0.5 if dtype == torch.int8 else t.abs() * 2.0 ** -4
    assert bool(((q.float().double() - t).abs() <= step).all()), q.float().tolist()


def test_codes_as_bytes_are_e4m3():
    """uint8 stands for e4m3 bytes, as it does in every call that takes codes; other types are refused."""
    v = torch.randn(5, 70, generator=torch.Generator().manual_seed(2))
    want, s0 = q8.quantise_rows(v, torch.float8_e4m3fn)
    q, s = q8.quantise_rows(v, torch.uint8)
    assert q.dtype == torch.uint8 and q.stride() == want.stride()
    assert torch.equal(q, want.view(torch.uint8)) and torch.equal(s, s0)
    for dtype in (torch.float16, torch.int32, torch.float8_e5m2):
        with pytest.raises(ValueError):
            q8.quantise_rows(v, dtype)


def test_codes_do_not_depend_on_the_default_type():
    v = torch.randn(3, 40, generator=torch.Generator().manual_seed(3))
    v[1] *= 1e-43
    want = q8.quantise_rows(v)
    torch.set_default_dtype(torch.float16)
    try:
        got = q8.quantise_rows(v)
    finally:
        torch.set_default_dtype(torch.float32)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
