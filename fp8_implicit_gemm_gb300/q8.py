"""The quantised transformer operators of ``include/q8.h`` and ``include/q8_attention.h`` as a program
uses them: a linear layer that owns its weights' codes and its plan, a gated MLP block made of the
three operators, and what attention takes: rotations, a paged cache of codes, attention over it and
over prompts, and a block that makes one layer's attention of them.

    python -m fp8_implicit_gemm_gb300.q8        # the blocks on random weights, against fp32
"""
from __future__ import annotations

import math

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


class Rotary:
    """The rotation of rot_dim elements of each head: pair j turns by frequency j times the token's position on
    the pair's axis. With sections (pairs for each axis, in order) each axis has its own frequencies
    theta^(-i / n) over its n pairs; without, there is one axis. `frequencies` (radians a position, rot_dim / 2
    of them) replaces those. Pairs are neighbours if `adjacent`, else half of rot_dim apart."""

    def __init__(self, rot_dim: int, theta: float = 10000.0, sections=None, adjacent: bool = False,
                 frequencies=None, device="cuda"):
        pairs = rot_dim // 2
        sections = [pairs] if sections is None else [int(n) for n in sections]
        if rot_dim < 2 or rot_dim % 2 or sum(sections) != pairs or min(sections) < 0:
            raise ValueError(f"expected an even rot_dim and sections of {pairs} pairs, got {rot_dim}, {sections}")
        if len(sections) > 4:
            raise ValueError(f"expected sections of up to 4 axes, got {sections}")
        if frequencies is None:
            frequencies = [theta ** -(i / n) for n in sections for i in range(n)]
        frequencies = [float(f) for f in frequencies]
        if len(frequencies) != pairs or not all(math.isfinite(f) for f in frequencies):
            raise ValueError(f"expected {pairs} finite frequencies")
        # turns a position in units of 2^-64, whole turns left out
        turns = [round(math.fmod(f / (2.0 * math.pi), 1.0) * 2.0 ** 64) % 2 ** 64 for f in frequencies]
        self.rot_dim, self.axes, self.adjacent = rot_dim, len(sections), bool(adjacent)
        self._turns = torch.tensor([t - 2 ** 64 if t >= 2 ** 63 else t for t in turns], dtype=torch.int64,
                                   device=device)
        axis = [a for a, n in enumerate(sections) for _ in range(n)]
        self._axis = torch.tensor(axis, dtype=torch.uint8, device=device)
        if self._turns.is_cuda:  # in place for calls on every stream
            torch.cuda.current_stream(self._turns.device).synchronize()
        self.table = (self._turns.data_ptr(), self._axis.data_ptr(), rot_dim, self.axes, int(self.adjacent),
                      self._turns.get_device())


class CacheQ8:
    """Keys and values of a layer as codes in pages (the layout of include/q8_attention.h). The tensors may be
    the caller's: 8-bit codes with scales [pages, kv_heads, page_size], or 4-bit codes, two in a byte, with
    scales [.., 2]. capi.heads_q8_run writes it, `read` gives rows back, CacheAttention attends over it."""

    def __init__(self, k_codes: torch.Tensor, k_scale: torch.Tensor, v_codes: torch.Tensor,
                 v_scale: torch.Tensor):
        self.k_codes, self.k_scale = k_codes.detach(), k_scale.detach()
        self.v_codes, self.v_scale = v_codes.detach(), v_scale.detach()
        self.parts = capi.cache_q8(self.k_codes, self.k_scale, self.v_codes, self.v_scale)
        self.pages, self.kv_heads, self.page_size, _ = k_codes.shape
        self.head_dim, self.code_type = self.parts[2], self.parts[3]

    @classmethod
    def empty(cls, pages: int, page_size: int, kv_heads: int, head_dim: int, codes=torch.int8,
              device="cuda") -> "CacheQ8":
        """A cache of zeros; `codes` is torch.int8, torch.float8_e4m3fn, or 4 for 4-bit codes."""
        if codes != 4:
            capi.q8_code_type(codes)
        shape = (pages, kv_heads, page_size)
        width, dtype = (head_dim // 2, torch.uint8) if codes == 4 else (head_dim, codes)
        c = [torch.zeros(shape + (width,), dtype=torch.uint8, device=device).view(dtype) for _ in "kv"]
        s = [torch.zeros(shape + (2,) * (codes == 4), dtype=torch.float32, device=device) for _ in "kv"]
        if c[0].is_cuda:  # in place for calls on every stream
            torch.cuda.current_stream(c[0].device).synchronize()
        return cls(c[0], s[0], c[1], s[1])

    def read(self, slots: torch.Tensor, k: torch.Tensor, v: torch.Tensor, stream=None) -> None:
        """k and v [tokens, kv_heads, head_dim] = the values at the slots [tokens] (int64)."""
        capi.cache_q8_read_run(self.parts, slots, k, v, stream)


class CacheAttention:
    """Attention of the newest tokens of up to max_seqs sequences over a cache. Owns a plan: one call at a
    time."""

    def __init__(self, cache: CacheQ8, q_heads: int, max_seqs: int = 256, max_tokens: int = 1,
                 scale: float | None = None):
        self._plan = 0
        self.cache, self.scale = cache, cache.head_dim ** -0.5 if scale is None else scale
        self._plan = capi.attn_q8_plan(max_seqs, max_tokens, q_heads, cache.kv_heads, cache.head_dim,
                                       cache.code_type, cache.parts[4])

    def __call__(self, q: torch.Tensor, table: torch.Tensor, lengths: torch.Tensor, o: torch.Tensor,
                 stream=None) -> torch.Tensor:
        """q, o: [seqs * tokens, q_heads, head_dim]; table: [seqs, width] pages, int32; lengths: [seqs], int32,
        the newest tokens, whose rows are in the cache already, included."""
        seqs = table.shape[0]
        capi.attn_q8_run(self._plan, q, self.cache.parts, table, lengths, o, self.scale,
                         q.shape[0] // seqs if seqs else 1, stream)
        return o

    def check(self) -> int:
        return capi.attn_q8_check(self._plan)

    def close(self) -> None:
        plan, self._plan = self._plan, 0
        capi.attn_q8_destroy(plan)

    def __del__(self):
        try:
            self.close()
        except Exception:  # the interpreter is ending and the library's module is gone
            pass


class PromptAttention:
    """Attention over whole prompts, packed one behind the other. Owns a plan, whose runs may be in flight
    at once."""

    def __init__(self, scale: float | None = None, device: int | None = None):
        self._plan = 0
        self.scale = scale
        self._plan = capi.attn_prompt_plan(torch.cuda.current_device() if device is None else device)

    def __call__(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, starts: torch.Tensor, o: torch.Tensor,
                 causal: bool = True, key_starts: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """q, o: [rows, q_heads, head_dim]; k, v: [key rows, kv_heads, head_dim]; starts: [seqs + 1] int32, of
        the keys too unless key_starts is given."""
        scale = q.shape[2] ** -0.5 if self.scale is None else self.scale
        capi.attn_prompt_run(self._plan, q, k, v, starts, o, scale, causal, key_starts, stream)
        return o

    def check(self) -> int:
        return capi.attn_prompt_check(self._plan)

    def close(self) -> None:
        plan, self._plan = self._plan, 0
        capi.attn_prompt_destroy(plan)

    def __del__(self):
        try:
            self.close()
        except Exception:  # the interpreter is ending and the library's module is gone
            pass


class AttentionQ8:
    """A layer's attention on 8-bit codes and a paged cache, up to its output product:

        residual += x;  a = norm(residual);  q, k, v = a * w_qkv^T, in heads;  q, k = their norms, turned;
        k and v to the cache;  o = attention

    for prompts (over their own keys in 16 bits; heads of up to 128) and for the newest tokens of running sequences
    (over the cache): four calls of the library either way, in the caller's buffers and its own, one call at a time.
    w_qkv [(q_heads + 2 * kv_heads) * head_dim, dim] holds the heads of q, then k's, then v's; the norms'
    weights [head_dim] and the rotary may be missing."""

    def __init__(self, norm_weight, w_qkv, q_heads, cache: CacheQ8, rotary: Rotary | None = None, q_norm=None,
                 k_norm=None, max_rows=8192, max_seqs=256, max_tokens=1, codes=torch.int8, eps=1e-6):
        kv, head_dim = cache.kv_heads, cache.head_dim
        rows, dim = w_qkv.shape
        if rows != (q_heads + 2 * kv) * head_dim or norm_weight.shape != (dim,):
            raise ValueError(f"expected norm_weight [dim] and w_qkv [{(q_heads + 2 * kv) * head_dim}, dim], got "
                             f"{tuple(norm_weight.shape)} and {tuple(w_qkv.shape)}")
        norms = [w for w in (q_norm, k_norm) if w is not None]
        if any(w.shape != (head_dim,) or w.dtype != norms[0].dtype for w in norms):
            raise ValueError(f"expected q_norm and k_norm [{head_dim}] of one type")
        device = w_qkv.get_device()
        if device < 0 or cache.parts[4] != device or norm_weight.get_device() != device:
            raise ValueError("expected norm_weight, w_qkv and the cache on one CUDA device")
        for w in norms:  # as the heads take them, after the residual has changed
            capi._q8_value_type(w, "q_norm, k_norm")
            capi._q8_vector(w, "q_norm, k_norm", head_dim, device)
        if rotary is not None and (rotary.rot_dim > head_dim or rotary.table[5] != device):
            raise ValueError(f"expected a rotary of up to {head_dim} elements on CUDA device {device}, got "
                             f"{rotary.rot_dim} on {rotary.table[5]}")
        if norm_weight.dtype not in (torch.bfloat16, torch.float16):  # the heads' type, which attention takes
            raise ValueError(f"expected a norm_weight of bfloat16 or float16, got {norm_weight.dtype}")
        self.norm_weight, self.eps, self.max_rows = norm_weight, eps, max_rows
        self.cache, self.rotary, self.q_norm, self.k_norm = cache, rotary, q_norm, k_norm
        self.qkv = LinearQ8(*quantise_rows(w_qkv, codes), max_rows=max_rows)
        self.newest = CacheAttention(cache, q_heads, max_seqs, max_tokens)
        dev = w_qkv.device
        self.prompts = PromptAttention(device=dev.index)
        torch.cuda.current_stream(dev).synchronize()  # the codes are in place for calls on every stream
        self._a = empty_codes(max_rows, dim, codes, dev)
        self._scale = torch.empty(max_rows, dtype=torch.float32, device=dev)
        self._qkv = torch.empty(max_rows, q_heads + 2 * kv, head_dim, dtype=norm_weight.dtype, device=dev)
        self._heads, self._dim, self._newest = (q_heads, kv, head_dim), dim, (max_seqs, max_tokens)

    def _start(self, x, residual, positions, slots, o, keep_keys, stream):
        rows, (heads, kv, head_dim) = x.shape[0], self._heads
        if rows > self.max_rows:
            raise ValueError(f"{rows} rows, planned for up to {self.max_rows}")
        # what the later calls take is refused here, before the first one has updated the residual
        device = x.get_device()
        address, pitch, head_pitch = capi._heads(o, "o", (rows, heads, head_dim), self._qkv.dtype, device)
        pitch, head_pitch = pitch if rows > 1 else heads * head_pitch, head_pitch if heads > 1 else head_dim
        apart = (pitch >= (heads - 1) * head_pitch + head_dim and head_pitch >= head_dim
                 or head_pitch >= (rows - 1) * pitch + head_dim and pitch >= head_dim)
        if rows and (address % 16 or pitch % 8 or head_pitch % 8 or not apart):
            raise ValueError("o: expected heads on 16 bytes that do not overlap")
        capi._q8_vector(slots, "slots", rows, device, torch.int64)
        if self.rotary is not None:
            if positions is None:
                raise ValueError("positions: expected with a rotary")
            want = (rows,) if self.rotary.axes == 1 and positions.dim() == 1 else (self.rotary.axes, rows)
            if (positions.shape != want or positions.dtype != torch.int64 or positions.get_device() != device
                    or (rows > 1 and positions.stride(-1) != 1) or (positions.dim() == 2 and 0 < positions.stride(0) < rows)):
                raise ValueError(f"positions: expected {want}, int64, on CUDA device {device}")
        a, scale, qkv = self._a[:rows], self._scale[:rows], self._qkv[:rows]
        capi.rmsnorm_q8_run(x, self.norm_weight, a, scale, self.eps, residual=residual, residual_out=residual,
                            stream=stream)
        self.qkv(a, scale, qkv.view(rows, -1), stream)
        q, k, v = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
        capi.heads_q8_run(q=q, q_out=q, k=k, k_out=k if keep_keys else None, v=v, q_weight=self.q_norm,
                          k_weight=self.k_norm, eps=self.eps, rotary=self.rotary,
                          positions=None if self.rotary is None else positions, cache=self.cache.parts, slots=slots,
                          stream=stream)
        return q, k, v

    def prompt(self, x, residual, starts, positions, slots, o, stream=None) -> torch.Tensor:
        """Whole prompts, packed: x, residual [rows, dim] (residual is updated in place), starts [seqs + 1]
        int32, positions [rows] or [axes, rows] and slots [rows] int64, o [rows, q_heads, head_dim]."""
        if self.cache.head_dim > 128:  # refused before the residual and the cache change, as in _start
            raise ValueError(f"prompts: expected heads of up to 128 elements, got {self.cache.head_dim}")
        capi._q8_index(starts, "starts", x.get_device())
        if starts.dim() != 1 or not 1 <= starts.shape[0] <= 65537:
            raise ValueError(f"starts: expected [seqs + 1] of up to 65536 sequences, got {tuple(starts.shape)}")
        q, k, v = self._start(x, residual, positions, slots, o, True, stream)
        return self.prompts(q, k, v, starts, o, stream=stream)

    def decode(self, x, residual, positions, slots, table, lengths, o, stream=None) -> torch.Tensor:
        """The newest tokens of sequences, as many of each: x, residual [seqs * tokens, dim], table [seqs,
        width] and lengths [seqs] int32 (the newest tokens included), the rest as for prompts."""
        rows, seqs, device = x.shape[0], table.shape[0], x.get_device()
        capi._q8_index(table, "table", device)
        capi._q8_index(lengths, "lengths", device)
        if table.dim() != 2 or lengths.shape != (seqs,) or (rows % seqs if seqs else rows):
            raise ValueError(f"expected a table and lengths of as many sequences as divide {rows} rows")
        if seqs > self._newest[0] or rows > seqs * self._newest[1] or (seqs and (rows < seqs or table.shape[1] < 1)):
            raise ValueError(f"expected up to {self._newest[0]} sequences of 1 to {self._newest[1]} rows and a page, got "
                             f"{rows} rows and a table {tuple(table.shape)}")
        if seqs > 1 and table.stride(0) < table.shape[1]:
            raise ValueError("table: expected rows that do not overlap")
        q, _, _ = self._start(x, residual, positions, slots, o, False, stream)
        return self.newest(q, table, lengths, o, stream)

    def check(self) -> int:
        statuses = [part.check() for part in (self.qkv, self.newest, self.prompts)]  # each clears what it reports
        return next((s for s in statuses if s != capi.CONV3D_OK), capi.CONV3D_OK)

    def close(self) -> None:
        for part in (self.qkv, self.newest, self.prompts):
            part.close()


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
    _demo_attention()


def _demo_attention() -> None:
    dim, heads, kv, head_dim, page, rows = 4096, 32, 8, 128, 64, 500
    w = torch.randn((heads + 2 * kv) * head_dim, dim, device="cuda") / dim ** 0.5
    weight = torch.ones(dim, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(rows, dim, device="cuda").bfloat16()
    a = x.float() * torch.rsqrt(x.float().square().mean(dim=1, keepdim=True) + 1e-6)
    q, k, v = (a @ w.t()).view(rows, -1, head_dim).split([heads, kv, kv], dim=1)
    angle = torch.arange(rows, device="cuda").double()[:, None] * 10000.0 ** -(
        torch.arange(head_dim // 2, device="cuda", dtype=torch.float64) / (head_dim // 2))
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]

    def turned(t):
        z = torch.complex(*t.double().chunk(2, dim=-1)) * turn
        return torch.cat([z.real, z.imag], dim=-1).float()
    q, k = turned(q), turned(k)
    score = torch.einsum("ihgd,jhd->hgij", q.view(rows, kv, -1, head_dim), k) * head_dim ** -0.5
    score = score.masked_fill(torch.ones(rows, rows, dtype=torch.bool, device="cuda").triu(1), -torch.inf)
    want = torch.einsum("hgij,jhd->ihgd", score.softmax(dim=-1), v).reshape(rows, heads, head_dim)
    table = torch.arange(8, dtype=torch.int32, device="cuda")[None]
    at = torch.arange(rows, device="cuda")
    for codes, name in ((4, "4-bit"), (torch.int8, "int8"), (torch.float8_e4m3fn, "e4m3")):
        cache = CacheQ8.empty(8, page, kv, head_dim, codes)
        layer = AttentionQ8(weight, w, heads, cache, Rotary(head_dim), max_rows=rows)
        o = torch.empty(rows, heads, head_dim, dtype=torch.bfloat16, device="cuda")
        n = rows - 1  # the last token comes by itself, over the cache
        starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        layer.prompt(x[:n], torch.zeros_like(x[:n]), starts, at[:n], at[:n], o[:n])
        lengths = torch.tensor([rows], dtype=torch.int32, device="cuda")
        layer.decode(x[n:], torch.zeros_like(x[n:]), at[n:], at[n:], table, lengths, o[n:])
        assert layer.check() == capi.CONV3D_OK
        prompt, newest = [float((o[s].float() - want[s]).norm() / want[s].norm()) for s in (slice(n), slice(n, rows))]
        print(f"attention {dim} -> {heads} + 2 x {kv} heads of {head_dim}, int8 weights, {name} cache: relative "
              f"error against fp32 {prompt:.4f} (prompt of {n}), {newest:.4f} (the next token)")
        layer.close()


if __name__ == "__main__":
    _demo()
