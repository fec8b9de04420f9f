"""The C ABI of include/q8_attention.h, as far as it goes without a GPU: exports, struct layouts and the
refusals that come before any device access."""
import ctypes
import os
import re
import struct
import subprocess

import pytest
import torch

from fp8_implicit_gemm_gb300 import build, capi, q8

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "q8_attention.h")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return capi.load()


def test_library_exports_every_declared_symbol(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b((?:heads|cache|attn)_[a-z0-9_]+)\s*\(", text))
    assert {"heads_q8_run", "cache_q8_read_run", "attn_q8_plan", "attn_q8_plan_ex", "attn_q8_run", "attn_q8_check",
            "attn_q8_workspace_size", "attn_q8_destroy", "attn_prompt_plan", "attn_prompt_plan_ex",
            "attn_prompt_run", "attn_prompt_check", "attn_prompt_destroy"} == names
    for n in names:
        assert hasattr(lib, n), n


def test_packed_arguments_have_the_structs_layout(tmp_path):
    types = {"q8_cache": (capi._CACHE, ["pages", "page_size", "code_type"]),
             "heads_q8_args": (capi._HEADS_ARGS, ["slots", "cache", "q_pitch", "positions_pitch", "tokens",
                                                  "stream", "q_heads", "device", "eps"]),
             "cache_q8_read_args": (capi._CACHE_READ_ARGS, ["k_pitch", "tokens", "stream", "device"]),
             "attn_q8_args": (capi._ATTN_ARGS, ["lengths", "q_pitch", "table_pitch", "stream", "tokens",
                                                "scale"]),
             "attn_prompt_args": (capi._ATTN_PROMPT_ARGS, ["key_starts", "q_pitch", "seqs", "stream",
                                                           "q_heads", "scale"])}
    lines = [f'printf("%zu ", sizeof({t}));' for t in types]
    lines += [f'printf("%zu ", offsetof({t}, {f}));' for t, (_, fields) in types.items() for f in fields]
    src, exe = tmp_path / "s.c", tmp_path / "s"
    src.write_text('#include <stdio.h>\n#include "q8_attention.h"\nint main(void){' + "".join(lines) + "}\n")
    subprocess.run(["gcc", "-I", os.path.dirname(HEADER), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, check=True).stdout.split()]
    assert got[:5] == [s.size for s, _ in types.values()]
    assert got[5:] == [32, 40, 52, 80, 88, 96, 176, 184, 192, 200, 232, 236, 32, 64, 72, 84,
                       32, 40, 88, 96, 104, 116, 40, 48, 128, 136, 144, 164]


CACHE = dict(k_codes=4096, v_codes=4096, k_scale=4096, v_scale=4096, pages=8, page_size=16, kv_heads=2,
             head_dim=64, code_type=1)


def _cache(**kw):
    return ctypes.create_string_buffer(capi._CACHE.pack(*{**CACHE, **kw}.values()), capi._CACHE.size)


HEADS = dict(q=4096, q_out=4096, k=4096, k_out=4096, v=0, q_weight=4096, k_weight=4096, turns=4096, axis=0,
             positions=4096, slots=0, cache=0, q_pitch=256, q_head_pitch=64, q_out_pitch=256,
             q_out_head_pitch=64, k_pitch=128, k_head_pitch=64, k_out_pitch=128, k_out_head_pitch=64,
             v_pitch=128, v_head_pitch=64, positions_pitch=16, tokens=4, stream=0, q_heads=4, kv_heads=2,
             head_dim=64, rot_dim=64, axes=1, adjacent=0, value_type=2, weight_type=2, device=0, eps=1e-6)


def _heads(cache=None, **kw):
    a = {**HEADS, **kw}
    held = None
    if cache is not None:
        held = _cache(**cache)
        a.update(cache=ctypes.addressof(held))
        a.setdefault("v", 4096)
    return capi.load().heads_q8_run(capi._HEADS_ARGS.pack(*a.values()))


@pytest.mark.parametrize("kw", [
    dict(q=0, q_out=0, k=0, k_out=0), dict(q_out=0), dict(q=0), dict(k_out=0), dict(k=0), dict(tokens=-1),
    dict(q=4104), dict(q_out=4098), dict(k=4100), dict(k_out=4104), dict(q_pitch=255), dict(q_pitch=252),
    dict(q_pitch=192), dict(q_head_pitch=60), dict(k_head_pitch=32), dict(k_out_pitch=64), dict(v=4096),
    dict(slots=4096), dict(q_weight=4097), dict(weight_type=0), dict(weight_type=1, k_weight=4098),
    dict(value_type=0), dict(value_type=4), dict(rot_dim=0), dict(rot_dim=63), dict(rot_dim=66), dict(axes=0),
    dict(axes=5), dict(axes=2), dict(axes=2, axis=4096, positions_pitch=3), dict(positions=0),
    dict(positions=4100), dict(turns=4100), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(head_dim=0), dict(q_heads=0), dict(kv_heads=0), dict(q=0, q_out=0), dict(k=0, k_out=0)])
def test_heads_refuse(lib, kw):
    assert _heads(**kw) == capi.CONV3D_EINVAL


@pytest.mark.parametrize("cache,kw", [
    (dict(), dict(v=4096)), (dict(), dict(slots=4096)), (dict(kv_heads=1), dict(v=4096, slots=4096)),
    (dict(head_dim=128), dict(v=4096, slots=4096)), (dict(page_size=24), dict(v=4096, slots=4096)),
    (dict(page_size=0), dict(v=4096, slots=4096)), (dict(pages=0), dict(v=4096, slots=4096)),
    (dict(code_type=4), dict(v=4096, slots=4096)), (dict(k_codes=0), dict(v=4096, slots=4096)),
    (dict(v_scale=4104), dict(v=4096, slots=4096)), (dict(), dict(v=4104, slots=4096)),
    (dict(), dict(v=4096, slots=4100)), (dict(), dict(v=4096, slots=4096, k=0, k_out=0, k_weight=0)),
    (dict(), dict(v=4096, slots=4096, v_head_pitch=32))])
def test_heads_refuse_with_a_cache(lib, cache, kw):
    assert _heads(cache, **kw) == capi.CONV3D_EINVAL


@pytest.mark.parametrize("kw", [
    dict(head_dim=68, q_head_pitch=72, k_head_pitch=72, rot_dim=64), dict(tokens=1 << 31), dict(q_heads=1 << 16),
    dict(head_dim=264, q_head_pitch=264)])
def test_heads_unsupported(lib, kw):
    assert _heads(**kw) == capi.CONV3D_EUNSUPPORTED


@pytest.mark.parametrize("cache", [dict(head_dim=80), dict(kv_heads=1 << 15), dict(pages=1 << 27)])
def test_caches_unsupported(lib, cache):
    assert _heads(cache, v=4096, slots=4096) == capi.CONV3D_EUNSUPPORTED
    assert _read(cache) == capi.CONV3D_EUNSUPPORTED


def _read(fields=None, **kw):
    held = _cache(**(fields or {}))
    a = dict(cache=ctypes.addressof(held), slots=4096, k=4096, v=4096, k_pitch=128, k_head_pitch=64, v_pitch=128,
             v_head_pitch=64, tokens=4, stream=0, value_type=2, device=0)
    a.update(kw)
    return capi.load().cache_q8_read_run(capi._CACHE_READ_ARGS.pack(*a.values()))


@pytest.mark.parametrize("kw", [dict(cache=0), dict(slots=0), dict(slots=4100), dict(k=0), dict(v=4104),
                                dict(k_pitch=64), dict(v_head_pitch=60), dict(tokens=-1), dict(value_type=9)])
def test_read_refuses(lib, kw):
    assert _read(**kw) == capi.CONV3D_EINVAL


def test_plans_refuse(lib):
    h = ctypes.c_void_p(1)
    for args in ((0, 1, 4, 2, 64, 1), (1, 0, 4, 2, 64, 1), (1, 1, 0, 2, 64, 1), (1, 1, 4, 0, 64, 1),
                 (1, 1, 4, 3, 64, 1), (1, 1, 4, 2, 0, 1), (1, 1, 4, 2, 64, 0), (1, 1, 4, 2, 64, 4)):
        h.value = 1
        assert lib.attn_q8_plan(ctypes.byref(h), *args, 0) == capi.CONV3D_EINVAL and h.value is None
    for args in ((1, 1, 4, 2, 80, 1), (65537, 1, 4, 2, 64, 1), (1, 65, 4, 2, 64, 1), (1, 1, 4096, 2, 64, 1)):
        assert lib.attn_q8_plan(ctypes.byref(h), *args, 0) == capi.CONV3D_EUNSUPPORTED
    assert lib.attn_q8_plan(None, 1, 1, 4, 2, 64, 1, 0) == capi.CONV3D_EINVAL
    assert lib.attn_prompt_plan(None, 0) == capi.CONV3D_EINVAL
    o = capi.AttnOptions(wait_timeout_ms=-1)
    assert lib.attn_prompt_plan_ex(ctypes.byref(h), 0, ctypes.byref(o)) == capi.CONV3D_EINVAL
    assert lib.attn_q8_plan_ex(ctypes.byref(h), 1, 1, 4, 2, 64, 1, 0, ctypes.byref(o)) == capi.CONV3D_EINVAL


def test_null_arguments(lib):
    assert lib.heads_q8_run(None) == lib.cache_q8_read_run(None) == capi.CONV3D_EINVAL
    assert lib.attn_q8_run(None, None) == lib.attn_prompt_run(None, None) == capi.CONV3D_EINVAL
    assert lib.attn_q8_check(None) == lib.attn_prompt_check(None) == capi.CONV3D_EINVAL
    assert lib.attn_q8_workspace_size(None) == 0
    lib.attn_q8_destroy(None)
    lib.attn_prompt_destroy(None)


def test_rotary_table():
    """Turns of 2^-64; signed storage of unsigned words; whole turns of fast frequencies left out."""
    import math
    r = q8.Rotary(8, theta=10000.0, device="cpu")
    assert r._turns.tolist() == [round(10000.0 ** -(i / 4) / (2 * math.pi) * 2.0 ** 64) for i in range(4)]
    r = q8.Rotary(8, sections=[1, 3], theta=100.0, device="cpu")
    assert r._axis.tolist() == [0, 1, 1, 1] and r.axes == 2
    assert r._turns.tolist()[0] == r._turns.tolist()[1]
    t = q8.Rotary(2, frequencies=[2 * math.pi * 5.75], device="cpu")._turns.item()
    assert abs(struct.unpack("Q", struct.pack("q", t))[0] / 2.0 ** 64 - 0.75) < 1e-14
    t = q8.Rotary(2, frequencies=[-2 * math.pi * 0.25], device="cpu")._turns.item()
    assert abs(t / 2.0 ** 64 + 0.25) < 1e-14
    for bad in (dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=8, sections=[1, 2]),
                dict(rot_dim=8, sections=[5, -1]), dict(rot_dim=4, frequencies=[1.0]),
                dict(rot_dim=4, frequencies=[1.0, float("inf")])):
        with pytest.raises(ValueError):
            q8.Rotary(device="cpu", **bad)


def test_python_refuses_what_is_not_on_a_gpu():
    x = torch.zeros(2, 4, 64)
    with pytest.raises(ValueError):
        capi.heads_q8_run(q=x, q_out=x)
    with pytest.raises(ValueError):
        capi.cache_q8(torch.zeros(1, 1, 16, 64, dtype=torch.int8), torch.zeros(1, 1, 16),
                      torch.zeros(1, 1, 16, 64, dtype=torch.int8), torch.zeros(1, 1, 16))
    with pytest.raises(ValueError):
        capi.attn_prompt_run(0, x, x, x, torch.zeros(2, dtype=torch.int32), x, 1.0)


def test_rotary_of_more_axes_than_the_heads_take():
    q8.Rotary(16, sections=[2, 2, 2, 2], device="cpu")
    with pytest.raises(ValueError):
        q8.Rotary(16, sections=[2, 2, 2, 1, 1], device="cpu")


class _Heads:
    """What the binding asks of a tensor, on a device that is not there."""

    def __init__(self, shape, dtype, device):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, device

    def get_device(self):
        return self.device

    def stride(self, dim=None):
        t = torch.empty(self.shape, device="meta")
        return t.stride() if dim is None else t.stride(dim)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096


@pytest.mark.parametrize("of_plan,of_tensors", [(0, 0), (0, 1), (1, 0)])
def test_attention_on_another_device_than_the_plans(lib, monkeypatch, of_plan, of_tensors):
    """Plans of one device with tensors of another are refused, whichever is the current one."""
    calls = []

    class Fake:
        def attn_q8_plan_ex(self, h, *args):
            h._obj.value = 64
            return 0

        def attn_prompt_plan_ex(self, h, *args):
            h._obj.value = 128
            return 0

        def attn_q8_run(self, *args):
            calls.append("cache")
            return 0

        def attn_prompt_run(self, *args):
            calls.append("prompt")
            return 0

        def attn_q8_destroy(self, plan):
            pass

        attn_prompt_destroy = attn_q8_destroy
    capi._q8_setup()
    fake = Fake()
    monkeypatch.setattr(capi, "_q8", fake)
    monkeypatch.setattr(capi, "load", lambda: fake)
    x = _Heads((2, 4, 64), torch.bfloat16, of_tensors)
    ints = [_Heads(shape, torch.int32, of_tensors) for shape in ((2,), (2, 1))]
    cache = (4096, 2, 64, capi.Q8_INT8, of_tensors, None)
    plans = capi.attn_q8_plan(4, 1, 4, 2, 64, capi.Q8_INT8, of_plan), capi.attn_prompt_plan(of_plan)
    runs = (lambda: capi.attn_q8_run(plans[0], x, cache, ints[1], ints[0], x, 1.0, stream=0),
            lambda: capi.attn_prompt_run(plans[1], x, x, x, ints[0], x, 1.0, stream=0))
    for run in runs:
        if of_plan == of_tensors:
            run()
        else:
            with pytest.raises(ValueError):
                run()
    assert calls == (["cache", "prompt"] if of_plan == of_tensors else [])
    capi.attn_q8_destroy(plans[0])
    capi.attn_prompt_destroy(plans[1])
    again = capi.attn_prompt_plan(of_tensors)  # the same handle, of another device now
    capi.attn_prompt_run(again, x, x, x, ints[0], x, 1.0, stream=0)
    capi.attn_prompt_destroy(again)


@pytest.mark.parametrize("shape,codes,offset", [
    ((2, 2, 24, 64), torch.int8, 0), ((2, 2, 16, 80), torch.int8, 0), ((0, 2, 16, 64), torch.int8, 0),
    ((2, 0, 16, 64), torch.int8, 0), ((2, 2, 16, 512), torch.int8, 0), ((1 << 27, 1, 16, 64), torch.int8, 0),
    ((2, 1 << 15, 16, 64), torch.int8, 0), ((2, 2, 16, 64), torch.int8, 8), ((2, 2, 16, 64), torch.uint8, 4),
    ((2, 2, 16, 24), torch.uint8, 0)])
def test_caches_that_no_call_takes(lib, shape, codes, offset):
    """They are refused where a cache is made, so that no block finds out after it has updated a residual."""
    class Tensor(_Heads):
        def dim(self):
            return len(self.shape)

        def data_ptr(self):
            return 4096 + offset
    four = codes == torch.uint8
    c = Tensor(shape, codes, 0)
    scale = Tensor(shape[:3] + (2,) * four, torch.float32, 0)
    with pytest.raises(ValueError):
        capi.cache_q8(c, scale, c, scale)
    good = Tensor((2, 2, 16, 64), codes, 0)
    good.data_ptr = lambda: 4096
    scale = Tensor((2, 2, 16) + (2,) * four, torch.float32, 0)
    scale.data_ptr = good.data_ptr
    assert capi.cache_q8(good, scale, good, scale)[1:5] == (2, 128 if four else 64, capi.Q8_INT4 if four else capi.Q8_INT8, 0)
