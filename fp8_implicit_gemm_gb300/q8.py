"""The 8-bit transformer operators of ``include/q8.h`` as a program uses them: a linear layer that
owns its weights' codes and its plan, and a gated MLP block made of the three operators.

    python -m fp8_implicit_gemm_gb300.q8        # one block on random weights, against fp32
"""
from __future__ import annotations

import torch

from . import capi


def empty_codes(rows: int, cols: int, dtype=torch.int8, device="cuda") -> torch.Tensor:
    """An uninitialised [rows, cols] matrix of codes whose row pitch is a multiple of 32 bytes. The
    linear layers take multiples of 16, but a row that starts inside a 32-byte sector costs them a
    sector more for every 128 codes: 4096 x 8192 x 1001 e4m3 takes 56 us with both matrices on 16
    bytes, 40 on 32."""
    return torch.empty(rows, -(-cols // 32) * 32, dtype=dtype, device=device)[:, :cols]


def quantise_rows(v: torch.Tensor, dtype=torch.int8) -> tuple[torch.Tensor, torch.Tensor]:
    """Codes and scales of a matrix's rows by torch operations, for weights, which are laid out
    once (a step's activations get theirs from the norm or the activation). A row that is not
    finite gets the scale NaN and codes 0, as it does there."""
    if capi.q8_code_type(dtype) == capi.Q8_E4M3 and dtype != torch.float8_e4m3fn:  # e4m3 bytes
        q, scale = quantise_rows(v, torch.float8_e4m3fn)
        return q.view(dtype), scale
    top = 127.0 if dtype == torch.int8 else 448.0
    v = v.float()
    amax = v.abs().amax(dim=1)
    scale = torch.where(amax > 0, amax / top, torch.ones_like(amax))
    finite = torch.isfinite(amax)
    q = empty_codes(*v.shape, dtype=dtype, device=v.device)
    # a row so small that its scale rounds coarsely, or to 0, is lifted for its quotients
    lift = torch.ones_like(amax).masked_fill_((amax > 0) & (amax < 2.0 ** -100), 2.0 ** 100)
    by = torch.where(amax > 0, amax * lift / top, torch.ones_like(amax))
    v = torch.where(finite[:, None], v * lift[:, None] / by[:, None], 0.0)
    scale = torch.where(finite, scale, torch.nan)
    q.copy_(v.round() if dtype == torch.int8 else v.clamp(-top, top))
    return q, scale


class LinearQ8:
    """y = (x * w^T) scaled by token and channel, plus a bias. Owns a plan for up to max_rows tokens
    and keeps the weights' codes (copied once if their rows do not lie on 32-byte boundaries, as the
    kernels read them fastest: what the caller changes in its own tensor later then does not reach the
    layer; scales and bias, and codes laid out so, stay the caller's memory). One call at a time: a
    plan's workspace is shared by its runs. For int8 codes it takes 2 * max_rows * K bytes."""

    def __init__(self, w: torch.Tensor, scale_w: torch.Tensor, bias: torch.Tensor | None = None,
                 max_rows: int = 8192):
        self._plan = 0
        if w.stride(1) != 1 or w.stride(0) % 32 or w.data_ptr() % 32:
            w = empty_codes(*w.shape, dtype=w.dtype, device=w.device).copy_(w)
            if w.is_cuda:  # in place for calls on every stream
                torch.cuda.current_stream(w.device).synchronize()
        # tensors of its own on the same memory: what the caller does to its own ones later frees none
        # of what the calls read
        self.w, self.scale_w = w.detach(), scale_w.detach()
        self.bias = None if bias is None else bias.detach()
        self._weights = capi.linear_q8_weights(self.w, self.scale_w, self.bias)
        self.max_rows = max_rows
        self._plan = capi.linear_q8_plan(max_rows, w.shape[0], w.shape[1],
                                         capi.q8_code_type(w.dtype), w.get_device())

    def __call__(self, x: torch.Tensor, scale_x: torch.Tensor, y: torch.Tensor,
                 stream=None) -> torch.Tensor:
        capi.linear_q8_run_weights(self._plan, x, scale_x, self._weights, y, stream)
        return y

    def check(self) -> int:
        return capi.linear_q8_check(self._plan)

    def close(self) -> None:
        plan, self._plan = self._plan, 0
        capi.linear_q8_destroy(plan)

    def __del__(self):
        try:
            self.close()
        except Exception:  # the interpreter is ending and the library's module is gone
            pass


class MlpQ8:
    """A transformer's gated MLP on 8-bit codes:

        residual += x;  a = norm(residual);  g, u = a * w_gate_up^T;  y = (silu(g) * u) * w_down^T

    four calls of the library, in the caller's buffers and its own (made once): as many launches, and one
    more for each product of int8 codes on the tensor cores."""

    def __init__(self, norm_weight, w_gate_up, w_down, max_rows=8192, codes=torch.int8, eps=1e-6):
        dim, inner = w_down.shape
        if w_gate_up.shape != (2 * inner, dim) or norm_weight.shape != (dim,):
            raise ValueError("expected norm_weight [dim], w_gate_up [2 * inner, dim], "
                             "w_down [dim, inner]")
        self.norm_weight, self.eps, self.max_rows = norm_weight, eps, max_rows
        self.gate_up = LinearQ8(*quantise_rows(w_gate_up, codes), max_rows=max_rows)
        self.down = LinearQ8(*quantise_rows(w_down, codes), max_rows=max_rows)
        dev = w_down.device
        torch.cuda.current_stream(dev).synchronize()  # the codes are in place for calls on every stream
        self._a = empty_codes(max_rows, dim, codes, dev)
        self._h = empty_codes(max_rows, inner, codes, dev)
        self._scale_a = torch.empty(max_rows, dtype=torch.float32, device=dev)
        self._scale_h = torch.empty(max_rows, dtype=torch.float32, device=dev)
        self._gu = torch.empty(max_rows, 2 * inner, dtype=norm_weight.dtype, device=dev)
        self._inner = inner

    def __call__(self, x: torch.Tensor, residual: torch.Tensor, y: torch.Tensor,
                 stream=None) -> torch.Tensor:
        """x, residual, y: [rows, dim]; residual is updated in place, y is returned."""
        rows = x.shape[0]
        if rows > self.max_rows:
            raise ValueError(f"{rows} rows, planned for up to {self.max_rows}")
        # y is the last call's argument: refused here, before the first one has updated the residual
        capi._q8_pitch(y, "y", x.shape, x.get_device())
        capi._q8_value_type(y, "y")
        a, scale_a, gu = self._a[:rows], self._scale_a[:rows], self._gu[:rows]
        h, scale_h = self._h[:rows], self._scale_h[:rows]
        capi.rmsnorm_q8_run(x, self.norm_weight, a, scale_a, self.eps, residual=residual,
                            residual_out=residual, stream=stream)
        self.gate_up(a, scale_a, gu, stream)
        capi.silu_mul_q8_run(gu[:, :self._inner], gu[:, self._inner:], h, scale_h, stream)
        return self.down(h, scale_h, y, stream)

    def check(self) -> int:
        first, second = self.gate_up.check(), self.down.check()  # each clears what it reports
        return first or second

    def close(self) -> None:
        self.gate_up.close()
        self.down.close()


def _demo() -> None:
    torch.manual_seed(0)
    dim, inner, rows = 4096, 8192, 64
    w_gu = torch.randn(2 * inner, dim, device="cuda") / dim ** 0.5
    w_down = torch.randn(dim, inner, device="cuda") / inner ** 0.5
    weight = torch.ones(dim, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(rows, dim, device="cuda").bfloat16()
    h = x.float()
    a = h * torch.rsqrt(h.square().mean(dim=1, keepdim=True) + 1e-6)
    g, u = (a @ w_gu.t()).chunk(2, dim=1)
    want = (torch.nn.functional.silu(g) * u) @ w_down.t()
    for codes in (torch.int8, torch.float8_e4m3fn):
        mlp = MlpQ8(weight, w_gu, w_down, max_rows=rows, codes=codes)
        y = mlp(x, torch.zeros_like(x), torch.empty_like(x))
        assert mlp.check() == capi.CONV3D_OK
        err = float((y.float() - want).norm() / want.norm())
        print(f"gated MLP {dim} -> {inner} -> {dim}, {rows} tokens, {codes}: "
              f"relative error against fp32 weights {err:.4f}")
        mlp.close()


if __name__ == "__main__":
    _demo()
