"""The C ABI of include/q8.h, as far as it goes without a GPU: exports, struct layouts and the
refusals that come before any device access."""
import ctypes
import os
import re
import subprocess

import pytest

from fp8_implicit_gemm_gb300 import build, capi

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "q8.h")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return capi.load()


def test_library_exports_every_declared_symbol(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b((?:rmsnorm|silu_mul|linear)_q8_[a-z_]+)\s*\(", text))
    assert {"rmsnorm_q8_run", "silu_mul_q8_run", "linear_q8_plan", "linear_q8_run",
            "linear_q8_check", "linear_q8_destroy", "linear_q8_workspace_size"} <= names
    for n in names:
        assert hasattr(lib, n), n


def test_packed_arguments_have_the_structs_layout(tmp_path):
    fields = {"rmsnorm_q8_args": ["rows", "stream", "value_type", "device", "eps"],
              "silu_mul_q8_args": ["rows", "stream", "value_type", "device"],
              "linear_q8_args": ["rows", "N", "K", "stream", "y_type", "code_type"]}
    lines = [f'printf("%zu\\n", sizeof({t}));' for t in fields]
    lines += [f'printf("%zu\\n", offsetof({t}, {f}));' for t in fields for f in fields[t]]
    src, exe = tmp_path / "s.c", tmp_path / "s"
    src.write_text('#include <stdio.h>\n#include "q8.h"\nint main(void){' + "".join(lines) + "}\n")
    subprocess.run(["gcc", "-I", os.path.dirname(HEADER), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, check=True).stdout.split()]
    assert got[:3] == [capi._RMSNORM_ARGS.size, capi._SILU_MUL_ARGS.size, capi._LINEAR_ARGS.size]
    assert got[3:] == [80, 96, 104, 116, 120, 56, 72, 80, 88, 72, 80, 88, 96, 104, 112]


def _norm(**kw):
    a = dict(x=4096, residual=0, weight=4096, residual_out=0, q=4096, scale=4096, x_pitch=64,
             residual_pitch=64, residual_out_pitch=64, q_pitch=64, rows=4, cols=64, stream=0,
             value_type=1, weight_type=1, code_type=1, device=0, eps=1e-6, reserved=0)
    a.update(kw)
    return capi.load().rmsnorm_q8_run(capi._RMSNORM_ARGS.pack(*a.values()))


def _act(**kw):
    a = dict(gate=4096, up=4096, q=4096, scale=4096, gate_pitch=64, up_pitch=64, q_pitch=64, rows=4,
             cols=64, stream=0, value_type=1, code_type=1, device=0, reserved=0)
    a.update(kw)
    return capi.load().silu_mul_q8_run(capi._SILU_MUL_ARGS.pack(*a.values()))


@pytest.mark.parametrize("kw", [
    dict(x=0), dict(weight=0), dict(q=0), dict(scale=0), dict(rows=-1), dict(cols=0),
    dict(x_pitch=63), dict(q_pitch=63), dict(x=4098), dict(weight=4097), dict(scale=4097),
    dict(residual=4096), dict(residual_out=4096), dict(value_type=0), dict(value_type=4),
    dict(weight_type=0), dict(code_type=0), dict(code_type=3), dict(eps=-1.0),
    dict(eps=float("nan")), dict(eps=float("inf")),
    dict(residual=4096, residual_out=4096, residual_pitch=1),
    dict(residual=4096, residual_out=4096, residual_out_pitch=1),
    dict(residual=4098, residual_out=4096)])
def test_norm_refuses(lib, kw):
    assert _norm(**kw) == capi.CONV3D_EINVAL


@pytest.mark.parametrize("kw", [
    dict(gate=0), dict(up=0), dict(q=0), dict(scale=0), dict(rows=-1), dict(cols=0),
    dict(gate_pitch=63), dict(up_pitch=63), dict(q_pitch=63), dict(gate=4097), dict(scale=4098),
    dict(value_type=9), dict(code_type=9)])
def test_act_refuses(lib, kw):
    assert _act(**kw) == capi.CONV3D_EINVAL


def test_too_wide_is_unsupported(lib):
    wide = dict(cols=32769, q_pitch=32769)
    assert _norm(x_pitch=32769, **wide) == capi.CONV3D_EUNSUPPORTED
    assert _act(gate_pitch=32769, up_pitch=32769, **wide) == capi.CONV3D_EUNSUPPORTED


def test_null_arguments(lib):
    assert lib.rmsnorm_q8_run(None) == capi.CONV3D_EINVAL
    assert lib.silu_mul_q8_run(None) == capi.CONV3D_EINVAL
    assert lib.linear_q8_run(None, None) == capi.CONV3D_EINVAL
    assert lib.linear_q8_check(None) == capi.CONV3D_EINVAL
    assert lib.linear_q8_workspace_size(None) == 0
    lib.linear_q8_destroy(None)


def test_plan_refuses(lib):
    h = ctypes.c_void_p(1)
    for args in ((0, 64, 64, 1), (8, 0, 64, 1), (8, 64, 0, 1), (-1, 64, 64, 1), (8, 64, 64, 0),
                 (8, 64, 64, 3)):
        assert lib.linear_q8_plan(ctypes.byref(h), *args, 0) == capi.CONV3D_EINVAL
        assert h.value is None
    assert lib.linear_q8_plan(ctypes.byref(h), 1 << 30, 64, 64, 1, 0) == capi.CONV3D_EUNSUPPORTED
    assert lib.linear_q8_plan(None, 8, 64, 64, 1, 0) == capi.CONV3D_EINVAL
