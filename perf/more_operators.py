"""The operators of a quantised transformer's attention on real sizes: what each one is given, its plain
form, its calls in this package, and its value in 64 bits.

Five kinds of case ("op"):

  heads   every head of q and k: y = x / rms(x) * weight over the head, then rotated by its token's
          positions, one or several axes of them (capi.heads_q8_run)
  write   the same, with k and v left in a paged cache as codes; with "back" the rows are then read
          from the cache, as the next chunk of a prompt takes them (the same call, CacheQ8.read)
  read    rows of a cache as values                                              (CacheQ8.read)
  decode  softmax(q k^T) v for the newest tokens of sequences in a cache   (q8.CacheAttention)
  prompt  softmax(q k^T) v for packed sequences, grouped heads             (q8.PromptAttention)

Codes of a row (a token's head): int8 ("i8") or e4m3 ("e4m3") with scale = amax / 127 or 448 and the code
127 or 448 * value / amax; "i4" with scale = (highest - lowest) / 15 and the code 15 * (value - lowest) /
(highest - lowest), two in a byte, the first in the low bits; rounded to nearest even. A constant
row's scale is 1. (Quotients by the unrounded scale: 16-bit values lie on a tie often.)
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
TOP = {"i8": 127.0, "e4m3": 448.0}
CODE_TYPES = {"i8": torch.int8, "e4m3": torch.float8_e4m3fn, "i4": torch.uint8}
EPS = 1e-6
MOST_VALUES = 16384 * 32 * 128            # of a drawn case of the row operators: the largest listed one's
MOST_CACHE = 131072 * 8 * 128 * 2         # codes that a drawn decode reads
MOST_PRODUCT = 4.0 * 8192 * 8192 * 32 * 128  # of a drawn prompt, mask left aside


def listed():
    return [
        # one token of a running sequence, before attention: latency
        {"name": "heads 1 x 40 x 128", "op": "heads", "tokens": 1, "q_heads": 32, "kv_heads": 8,
         "dim": 128, "rot": 128, "axes": 1, "adjacent": False, "norm": True, "type": "bf16"},
        # the latents of a video block (16 x 64 x 64 in patches of 1 x 2 x 2): time, height, width
        {"name": "heads 16384 x 32 x 128 video", "op": "heads", "tokens": 16384, "q_heads": 16,
         "kv_heads": 16, "dim": 128, "rot": 128, "axes": 3, "adjacent": True, "norm": True,
         "type": "bf16"},
        # a ragged batch in 32 bits, half of a head rotated, no norm
        {"name": "heads 1501 x 16 x 80 f32", "op": "heads", "tokens": 1501, "q_heads": 12,
         "kv_heads": 4, "dim": 80, "rot": 40, "axes": 1, "adjacent": False, "norm": False,
         "type": "f32"},
        # eight sequences, one token each: norm, rotation and the cache in one call
        {"name": "write e4m3 8 x 40 x 128", "op": "write", "tokens": 8, "q_heads": 32, "kv_heads": 8,
         "dim": 128, "rot": 128, "axes": 1, "adjacent": False, "norm": True, "type": "bf16",
         "codes": "e4m3", "page": 64, "back": False},
        # a prompt's keys and values into a cache of 4 bits, and back for the next chunk
        {"name": "write i4 8192 x 8 x 128", "op": "write", "tokens": 8192, "q_heads": 0,
         "kv_heads": 8, "dim": 128, "rot": 0, "axes": 1, "adjacent": False, "norm": False,
         "type": "bf16", "codes": "i4", "page": 64, "back": True},
        # a long sequence's cache of 4 bits as values
        {"name": "read i4 65536 x 8 x 128", "op": "read", "tokens": 65536, "kv_heads": 8, "dim": 128,
         "codes": "i4", "page": 64, "type": "bf16"},
        # a short one of a small model, in 32 bits
        {"name": "read i8 777 x 5 x 64 f32", "op": "read", "tokens": 777, "kv_heads": 5, "dim": 64,
         "codes": "i8", "page": 16, "type": "f32"},
        # one sequence's next token: latency
        {"name": "decode i4 1 x 4096", "op": "decode", "seqs": 1, "longest": 4096, "ragged": False,
         "tokens": 1, "q_heads": 32, "kv_heads": 8, "dim": 128, "codes": "i4", "page": 64,
         "type": "bf16"},
        # a serving batch of sequences of all lengths: bandwidth
        {"name": "decode i4 64 x ..8192", "op": "decode", "seqs": 64, "longest": 8192,
         "ragged": True, "tokens": 1, "q_heads": 32, "kv_heads": 8, "dim": 128, "codes": "i4",
         "page": 64, "type": "bf16"},
        # one very long context in 8 bits
        {"name": "decode i8 1 x 131072", "op": "decode", "seqs": 1, "longest": 131072,
         "ragged": False, "tokens": 1, "q_heads": 64, "kv_heads": 8, "dim": 128, "codes": "i8",
         "page": 128, "type": "f16"},
        # a long prompt: the rate of the tensor cores
        {"name": "prompt 1 x 8192 causal", "op": "prompt", "seqs": 1, "longest": 8192,
         "ragged": False, "causal": True, "q_heads": 32, "kv_heads": 8, "dim": 128, "type": "bf16"},
        # sixteen short prompts of one small model, packed
        {"name": "prompt 16 x ..1000 x 64", "op": "prompt", "seqs": 16, "longest": 1000,
         "ragged": True, "causal": True, "q_heads": 14, "kv_heads": 2, "dim": 64, "type": "f16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["heads", "write", "read", "decode", "decode", "prompt", "prompt"])
    case = {"op": op, "type": rng.choice(["bf16", "bf16", "f16", "f32"]),
            "kv_heads": rng.choice([1, 2, 4, 5, 8, 16])}
    if op in ("heads", "write"):
        case["dim"] = rng.choice([64, 80, 96, 128, 128, 256])
        case["axes"] = rng.choice([1, 1, 2, 3])
        case["rot"] = case["dim"] if rng.random() < 0.7 else case["dim"] // 2
        case["adjacent"], case["norm"] = rng.random() < 0.4, rng.random() < 0.6
    if op in ("write", "read", "decode"):
        case["dim"] = rng.choice([64, 128, 128, 256])
        case["codes"] = rng.choice(["i4", "i4", "i8", "e4m3"])
        case["page"] = rng.choice([16, 32, 48, 64, 128, 256])
    if op in ("heads", "write", "read"):
        case["q_heads"] = 0 if op == "read" else case["kv_heads"] * rng.choice([1, 2, 4, 7, 8])
        heads = case["q_heads"] + 2 * case["kv_heads"]
        most = MOST_VALUES // (heads * case["dim"] * BYTES[case["type"]] // 2)
        case["tokens"] = _log(rng, 1, max(2, min(65536, most)))
    if op == "write":
        case["rot"] = case["dim"] if rng.random() < 0.7 else case["dim"] // 2
        case["back"] = case["codes"] != "e4m3"
        if case["type"] == "f32":
            case["type"] = "f16"
        if case["codes"] == "i4":  # keys that were rotated before
            case.update(q_heads=0, rot=0, axes=1, norm=False, adjacent=False)
    if op in ("decode", "prompt"):
        case["type"] = rng.choice(["bf16", "f16"])
        case["ragged"] = rng.random() < 0.6
        case["q_heads"] = case["kv_heads"] * rng.choice([1, 2, 4, 7, 8])
    if op == "decode":
        case["tokens"] = rng.choice([1, 1, 1, 2, 5])
        case["seqs"] = _log(rng, 1, 256)
        most = MOST_CACHE // (2 * case["seqs"] * case["kv_heads"] * case["dim"])
        case["longest"] = _log(rng, 16, max(17, min(131072, most)))
    if op == "prompt":
        case["dim"] = rng.choice([64, 80, 128, 128])
        case["causal"] = rng.random() < 0.7
        case["seqs"] = _log(rng, 1, 32)
        most = MOST_PRODUCT / (4.0 * case["seqs"] * case["q_heads"] * 128)
        case["longest"] = _log(rng, 1, max(2, min(16384, int(math.sqrt(most)))))
    return case


# ------------------------------------------------------------------------------------- inputs
def _values(gen, *shape):
    """Normal values, a few channels of each head of which are large, as keys and queries have them."""
    v = torch.randn(*shape, generator=gen, device=DEV)
    loud = torch.rand(shape[-2:], generator=gen, device=DEV) < 0.01
    return torch.where(loud, v * 6.0, v)


def _lengths(case):
    """Lengths of the sequences: equal ones, or spread evenly, the longest among them. The case's own."""
    if not case["ragged"]:
        return [case["longest"]] * case["seqs"]
    rng = random.Random(case["seqs"] * 1000003 + case["longest"])
    return [case["longest"]] + [rng.randint(1, case["longest"]) for _ in range(case["seqs"] - 1)]


def _shuffled(gen, case):
    n = torch.tensor(_lengths(case), device=DEV)
    return n[torch.randperm(len(n), generator=gen, device=DEV)]


def _pages(gen, count):
    """So many pages of a cache that holds some more, in no order."""
    total = count + 3
    return torch.randperm(total, generator=gen, device=DEV)[:count], total


def _slots(gen, case):
    """The slots of one sequence's tokens, and the cache's pages."""
    page = case["page"]
    pages, total = _pages(gen, -(-case["tokens"] // page))
    t = torch.arange(case["tokens"], device=DEV)
    return pages[t // page] * page + t % page, total


def _cache_codes(gen, pages, case):
    """A cache's codes and scales: normal keys and values quantised."""
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    out = {}
    for name in "kv":
        v = torch.randn(shape, generator=gen, device=DEV, dtype=torch.float16)
        q, scale = _plain_codes(v.float(), case["codes"])
        out[name + "_codes"], out[name + "_scale"] = _packed(q, case["codes"]), scale
    return out


def _empty_cache(pages, case):
    wide = case["dim"] // 2 if case["codes"] == "i4" else case["dim"]
    shape = (pages, case["kv_heads"], case["page"])
    out = {}
    for name in "kv":
        out[name + "_codes"] = torch.zeros(shape + (wide,), dtype=torch.uint8, device=DEV).view(
            CODE_TYPES[case["codes"]])
        out[name + "_scale"] = torch.zeros(shape + (2,) * (case["codes"] == "i4"), device=DEV)
    return out


def _sections(case):
    """Pairs of channels that turn by each axis: the first the time, a smaller share, then the others."""
    pairs = case["rot"] // 2
    if case["axes"] == 1:
        return [pairs]
    if case["axes"] == 2:
        return [pairs // 2, pairs - pairs // 2]
    rest = pairs * 3 // 8
    return [pairs - 2 * rest, rest, rest]


def _positions(gen, case):
    """A sequence's positions from somewhere in a long context, or a grid's coordinates."""
    t = torch.arange(case["tokens"], device=DEV)
    if case["axes"] == 1:
        return (t + torch.randint(0, 100000, (1,), generator=gen, device=DEV))[None]
    side = max(1, round(case["tokens"] ** (1 / 3)))
    grid = [t // (4 * side * side), t // (2 * side) % (2 * side), t % (2 * side)]
    return torch.stack(grid[3 - case["axes"]:])


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op, dim, kv, dtype = case["op"], case["dim"], case["kv_heads"], TYPES[case["type"]]
    s = {"case": case}
    if op in ("heads", "write"):
        heads, tokens = case["q_heads"], case["tokens"]
        # as one product leaves them
        x = _values(gen, tokens, heads + 2 * kv, dim).to(dtype)
        s["q"], s["k"], s["v"] = x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:]
        s["q_out"] = torch.empty(tokens, heads, dim, dtype=dtype, device=DEV)
        s["weights"] = [None, None]
        if case["norm"]:
            s["weights"] = list((1.0 + 0.1 * torch.randn(2, dim, generator=gen, device=DEV)).to(dtype))
        s["positions"] = _positions(gen, case)
        s["sections"] = _sections(case)
        # each axis has its own frequencies
        s["frequencies"] = torch.cat([10000.0 ** -(torch.arange(n, dtype=torch.float64) / n)
                                      for n in s["sections"]]).to(DEV)
        s["axis"] = torch.repeat_interleave(torch.arange(case["axes"]), torch.tensor(s["sections"])).to(DEV)
    if op == "heads":
        s["k_out"] = torch.empty(tokens, kv, dim, dtype=dtype, device=DEV)
    if op == "write":
        s["slots"], pages = _slots(gen, case)
        s["cache"] = _empty_cache(pages, case)
    if op == "read":
        s["slots"], pages = _slots(gen, case)
        s["cache"] = _cache_codes(gen, pages, case)
    if op == "read" or case.get("back"):
        s["k_back"], s["v_back"] = torch.empty(2, case["tokens"], kv, dim, dtype=dtype, device=DEV)
    if op == "decode":
        s["lengths"] = (_shuffled(gen, case) + (case["tokens"] - 1)).int()
        each = -(-(case["longest"] + case["tokens"] - 1) // case["page"])
        used, pages = _pages(gen, case["seqs"] * each)
        s["table"] = used.view(case["seqs"], each).int()
        s["cache"] = _cache_codes(gen, pages, case)
        s["q"] = (2.0 * torch.randn(case["seqs"] * case["tokens"], case["q_heads"], dim, generator=gen,
                                    device=DEV)).to(dtype)
        s["o"] = torch.empty_like(s["q"])
    if op == "prompt":
        n = _shuffled(gen, case)
        s["starts"] = torch.cat([n.new_zeros(1), n.cumsum(0)]).int()
        tokens = int(s["starts"][-1])
        s["q"] = (2.0 * torch.randn(tokens, case["q_heads"], dim, generator=gen, device=DEV)).to(dtype)
        s["k"], s["v"] = torch.randn(2, tokens, kv, dim, generator=gen, device=DEV).to(dtype)
        s["o"] = torch.empty_like(s["q"])
        s["longest"] = case["longest"]
    if own:  # the handles that a user's program keeps
        from fp8_implicit_gemm_gb300 import q8
        if op in ("heads", "write"):
            s["rotary"] = None
            if case["rot"]:
                s["rotary"] = q8.Rotary(case["rot"], sections=s["sections"], adjacent=case["adjacent"])
        if "cache" in s:
            s["paged"] = q8.CacheQ8(**s["cache"])
        if op == "decode":
            s["attend"] = q8.CacheAttention(s["paged"], case["q_heads"], max_seqs=case["seqs"],
                                            max_tokens=case["tokens"])
        if op == "prompt":
            s["attend"] = q8.PromptAttention()
    return s


# ------------------------------------------------------------------------------------- one pass
def _plain_codes(v, codes):
    """Codes as values of their own type (i4: 0 to 15) and scales of the rows along the last axis."""
    if codes == "i4":
        lowest, highest = v.amin(dim=-1), v.amax(dim=-1)
        width = torch.where(highest > lowest, highest - lowest, torch.full_like(lowest, 15.0))
        q = ((v - lowest[..., None]) * 15.0 / width[..., None]).round().to(torch.uint8)
        return q, torch.stack([width / 15.0, lowest], dim=-1)
    amax = v.abs().amax(dim=-1)
    amax = torch.where(amax > 0, amax, torch.full_like(amax, TOP[codes]))
    scale, v = amax / TOP[codes], v * TOP[codes] / amax[..., None]
    if codes == "i8":
        return v.round().clamp(-127.0, 127.0).to(torch.int8), scale
    return v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scale


def _packed(q, codes):
    return q[..., 0::2] | (q[..., 1::2] << 4) if codes == "i4" else q


def _plain_values(q, scale, codes):
    """fp32 values of packed codes."""
    if codes == "i4":
        q = torch.stack([q & 15, q >> 4], dim=-1).flatten(-2)
        return q.float() * scale[..., :1] + scale[..., 1:]
    return q.float() * scale[..., None]


def _plain_heads(s, x, weight):
    """x [tokens, heads, dim] normed and rotated, fp32."""
    x, case = x.float(), s["case"]
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + EPS) * weight.float()
    rot = case["rot"]
    if not rot:
        return x
    angle = s["positions"].double()[s["axis"]].t() * s["frequencies"]  # a far position's needs 64 bits
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if case["adjacent"] else (x[..., :rot // 2], x[..., rot // 2:rot])
    a, b = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([a, b], dim=-1).flatten(-2) if case["adjacent"] else torch.cat([a, b], dim=-1)
    return torch.cat([y, x[..., rot:]], dim=-1)


def _plain_write(s, name, v):
    case, cache = s["case"], s["cache"]
    q, scale = _plain_codes(v, case["codes"])
    page, at = s["slots"] // case["page"], s["slots"] % case["page"]
    as_bytes = cache[name + "_codes"].view(torch.uint8)
    as_bytes[page, :, at] = _packed(q, case["codes"]).view(torch.uint8)
    cache[name + "_scale"][page, :, at] = scale


def _plain_read(s, name):
    case, cache = s["case"], s["cache"]
    page, at = s["slots"] // case["page"], s["slots"] % case["page"]
    q = cache[name + "_codes"].view(torch.uint8)[page, :, at].view(CODE_TYPES[case["codes"]])
    v = _plain_values(q, cache[name + "_scale"][page, :, at], case["codes"])
    return v.to(s[name + "_back"].dtype)


def _plain_attention(q, k, v, seen):
    """softmax(q k^T) v over the keys that are seen; a row that sees none is 0. q [seqs, rows, heads,
    dim], k and v [seqs, keys, kv_heads, dim] in fp32, seen [seqs, rows, keys]."""
    seqs, rows, heads, dim = q.shape
    kv = k.shape[2]
    q = q.view(seqs, rows, kv, heads // kv, dim).permute(0, 2, 3, 1, 4)
    k, v = k.permute(0, 2, 1, 3)[:, :, None], v.permute(0, 2, 1, 3)[:, :, None]
    x = q @ k.transpose(-1, -2) * dim ** -0.5
    hidden = ~seen[:, None, None]
    x = x.masked_fill_(hidden, -torch.inf)
    top = x.amax(dim=-1, keepdim=True).clamp(min=-1e30)
    p = (x - top).exp_()
    o = p @ v / p.sum(dim=-1, keepdim=True).clamp(min=1e-30)
    return o.permute(0, 3, 1, 2, 4).reshape(seqs, rows, heads, dim)


def _plain_decode(s):
    case = s["case"]
    table, n = s["table"].long(), case["tokens"]
    kv, dim = case["kv_heads"], case["dim"]
    k, v = [_plain_values(s["cache"][name + "_codes"].view(torch.uint8)[table].view(CODE_TYPES[case["codes"]]),
                          s["cache"][name + "_scale"][table], case["codes"])
            .transpose(2, 3).reshape(case["seqs"], -1, kv, dim) for name in "kv"]
    at = torch.arange(k.shape[1], device=DEV)
    limit = s["lengths"][:, None].long() - n + 1 + torch.arange(n, device=DEV)
    seen = at < limit[:, :, None]
    q = s["q"].float().view(case["seqs"], n, case["q_heads"], dim)
    return _plain_attention(q, k, v, seen).reshape(s["q"].shape).to(s["o"].dtype)


def _padded(s):
    """Where the packed tokens lie in a batch of sequences padded to the longest."""
    starts = s["starts"].long()
    tokens = s["q"].shape[0]
    token = torch.arange(tokens, device=DEV)
    seq = torch.searchsorted(starts, token, right=True) - 1
    return seq, token - starts[seq], (s["case"]["seqs"], s["longest"])


def _plain_prompt(s):
    case = s["case"]
    seq, at, size = _padded(s)
    q, k, v = [torch.zeros(size + x.shape[1:], device=DEV).index_put_((seq, at), x.float())
               for x in (s["q"], s["k"], s["v"])]
    n = (s["starts"][1:] - s["starts"][:-1]).long()
    key = torch.arange(s["longest"], device=DEV)
    seen = (key < n[:, None])[:, None].expand(-1, s["longest"], -1)
    if case["causal"]:
        seen = seen & (key <= key[:, None])
    return _plain_attention(q, k, v, seen)[seq, at].to(s["o"].dtype)


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        from fp8_implicit_gemm_gb300 import capi
        if op in ("heads", "write"):
            capi.heads_q8_run(q=s["q"], q_out=s["q_out"], k=s["k"], k_out=s.get("k_out"),
                              v=s["v"] if op == "write" else None, q_weight=s["weights"][0],
                              k_weight=s["weights"][1], eps=EPS, rotary=s["rotary"],
                              positions=s["positions"] if s["rotary"] else None,
                              cache=s.get("paged"), slots=s.get("slots"))
        if op == "heads":
            return {"q": s["q_out"], "k": s["k_out"]}
        if op == "read" or s["case"].get("back"):
            s["paged"].read(s["slots"], s["k_back"], s["v_back"])
        if op == "decode":
            s["attend"](s["q"], s["table"], s["lengths"], s["o"])
        if op == "prompt":
            s["attend"](s["q"], s["k"], s["v"], s["starts"], s["o"], causal=s["case"]["causal"])
        return _outputs(s)
    if op in ("heads", "write"):
        q = _plain_heads(s, s["q"], s["weights"][0]).to(s["q_out"].dtype)
        k = _plain_heads(s, s["k"], s["weights"][1])
        if op == "heads":
            return {"q": q, "k": k.to(s["k_out"].dtype)}
        s["q_out"] = q
        _plain_write(s, "k", k)
        _plain_write(s, "v", s["v"].float())
    if op == "read" or s["case"].get("back"):
        s["k_back"], s["v_back"] = _plain_read(s, "k"), _plain_read(s, "v")
    if op == "decode":
        s["o"] = _plain_decode(s)
    if op == "prompt":
        s["o"] = _plain_prompt(s)
    return _outputs(s)


def _outputs(s):
    case = s["case"]
    if case["op"] in ("decode", "prompt"):
        return {"o": s["o"]}
    if case["op"] == "read":
        return {"k": s["k_back"], "v": s["v_back"]}
    r = {"q": s["q_out"]}
    if case["back"]:
        r.update(k=s["k_back"], v=s["v_back"])
    else:
        r.update(s["cache"])
    return r


# ------------------------------------------------------------------------------------- 64 bits
def _exact_e4m3(v):
    """v rounded to the nearest e4m3 value, ties to the even one: three bits behind the first, the
    smallest step 2^-9, the largest value 448."""
    mag = v.abs().clamp(max=448.0)
    _, power = torch.frexp(mag.clamp(min=2.0 ** -6))  # mag in [2^(power - 1), 2^power)
    step = torch.exp2(power.double() - 4)
    return torch.sign(v) * torch.clamp(torch.round(mag / step) * step, max=448.0)


def _exact_rows(v, codes):
    """What the codes of rows stand for: (codes, scale, lowest), each in 64 bits."""
    if codes == "i4":
        lowest = v.min(dim=-1, keepdim=True).values
        scale = (v.max(dim=-1, keepdim=True).values - lowest) / 15
        scale = torch.where(scale == 0, torch.ones_like(scale), scale)
        return torch.round((v - lowest) / scale), scale, lowest
    scale = v.abs().max(dim=-1, keepdim=True).values / TOP[codes]
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    q = torch.round(v / scale) if codes == "i8" else _exact_e4m3(v / scale)
    return q, scale, torch.zeros_like(scale)


def _exact_heads(s, x, weight):
    case, x = s["case"], x.double().clone()
    if weight is not None:
        x /= torch.sqrt(torch.sum(x * x, dim=-1, keepdim=True) / case["dim"] + EPS)
        x *= weight.double()
    half, first = case["rot"] // 2, 0
    for axis, n in enumerate(s["sections"] if half else []):
        for j in range(n):
            i = first + j
            a, b = (2 * i, 2 * i + 1) if case["adjacent"] else (i, i + half)
            turn = s["positions"][axis].double() * 10000.0 ** (-j / n)
            z = torch.complex(x[:, :, a], x[:, :, b]) * torch.polar(torch.ones_like(turn), turn)[:, None]
            x[:, :, a], x[:, :, b] = z.real, z.imag
        first += n
    return x


def _exact_sequence(q, k, v, limits):
    """One sequence and key head: q [rows, dim], k and v [keys, dim]; row i sees limits[i] keys."""
    if k.shape[0] == 0:
        return torch.zeros_like(q)
    x = torch.mm(q, k.t()) / math.sqrt(q.shape[1])
    x = torch.where(torch.arange(k.shape[0], device=DEV) < limits[:, None], x, -torch.inf)
    o = torch.mm(torch.softmax(x, dim=1), v)
    return torch.where(limits[:, None] > 0, o, torch.zeros_like(o))


def _exact_cached(cache, name, case, pages):
    """Values of one sequence's rows, [kv_heads, keys, dim] in 64 bits."""
    q, scale = cache[name + "_codes"][pages], cache[name + "_scale"][pages].double()
    if case["codes"] == "i4":
        v = torch.empty(q.shape[:-1] + (case["dim"],), dtype=torch.float64, device=DEV)
        v[..., 0::2], v[..., 1::2] = (q % 16).double(), (q // 16).double()
        v = v * scale[..., 0:1] + scale[..., 1:2]
    else:
        v = q.to(torch.float64) * scale.unsqueeze(-1)
    return v.transpose(0, 1).reshape(case["kv_heads"], -1, case["dim"])


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "heads":
        return {"q": _exact_heads(s, s["q"], s["weights"][0]), "k": _exact_heads(s, s["k"], s["weights"][1])}
    if op == "write":
        found = {"q": _exact_heads(s, s["q"], s["weights"][0])}
        rows = {"k": _exact_heads(s, s["k"], s["weights"][1]), "v": s["v"].double()}
        for name in "kv":
            q, scale, lowest = _exact_rows(rows[name], case["codes"])
            if case["back"]:
                found[name] = q * scale + lowest
                continue
            codes, scales = [torch.zeros_like(s["cache"][name + end], dtype=torch.float64)
                             for end in ("_codes", "_scale")]
            page = torch.div(s["slots"], case["page"], rounding_mode="floor")
            at = s["slots"] - page * case["page"]
            codes[page, :, at], scales[page, :, at] = q, scale.squeeze(-1)
            found[name + "_codes"], found[name + "_scale"] = codes, scales
        if not case["back"]:
            found = {"q": found["q"], **{name: found[name] for name in s["cache"]}}
        return found
    if op == "read":
        page = torch.div(s["slots"], case["page"], rounding_mode="floor")
        at = s["slots"] - page * case["page"]
        found = {}
        for name in "kv":
            v = _exact_cached(s["cache"], name, case, torch.arange(s["cache"]["k_codes"].shape[0], device=DEV))
            found[name] = v[:, page * case["page"] + at].transpose(0, 1)
        return found
    group = case["q_heads"] // case["kv_heads"]
    o = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    if case["seqs"] * case["kv_heads"] > 2048:
        return None
    for i in range(case["seqs"]):
        if op == "decode":
            n, length = case["tokens"], int(s["lengths"][i])
            at = i * n
            k, v = [_exact_cached(s["cache"], name, case, s["table"][i].long())[:, :length] for name in "kv"]
            limits = length - n + 1 + torch.arange(n, device=DEV)
        else:
            at, end = int(s["starts"][i]), int(s["starts"][i + 1])
            n = end - at
            k, v = [s[name][at:end].double().transpose(0, 1) for name in "kv"]
            limits = torch.arange(1, n + 1, device=DEV) if case["causal"] else torch.full((n,), n, device=DEV)
        for h in range(case["kv_heads"]):
            heads = slice(h * group, (h + 1) * group)
            q = s["q"][at:at + n, heads].double().reshape(n * group, -1)
            o[at:at + n, heads] = _exact_sequence(q, k[h], v[h], limits.repeat_interleave(group)).view(
                n, group, -1)
    return {"o": o}


# ------------------------------------------------------------------------------------- work
def _row_bytes(case):
    """Of a row of codes with its scale."""
    return case["dim"] // 2 + 8 if case["codes"] == "i4" else case["dim"] + 4


def work(case):
    """Each input read once, each output written once; the multiplications and additions."""
    op, dim, kv, size = case["op"], case["dim"], case["kv_heads"], BYTES[case["type"]]
    nbytes = flops = 0.0
    if op in ("heads", "write"):
        rows = case["tokens"] * (case["q_heads"] + kv)
        nbytes += rows * dim * size + case["tokens"] * 8 * case["axes"] + 2 * dim * size * case["norm"]
        flops += rows * (3.0 * case["rot"] + 5.0 * dim * case["norm"])
        nbytes += case["tokens"] * (case["q_heads"] + kv * (op == "heads")) * dim * size
    if op == "write":
        nbytes += case["tokens"] * (kv * dim * size + 8 + 2 * kv * _row_bytes(case))
        flops += 2 * case["tokens"] * kv * dim * 4.0
        if case["back"]:
            nbytes += case["tokens"] * 2 * kv * (dim * size + _row_bytes(case))
    if op == "read":
        nbytes += case["tokens"] * (2 * kv * (_row_bytes(case) + dim * size) + 8)
        flops += case["tokens"] * 2.0 * kv * dim
    if op == "decode":
        keys = sum(_lengths(case)) + case["seqs"] * (case["tokens"] - 1.0)
        nbytes += keys * 2 * kv * _row_bytes(case)
        nbytes += 2 * case["seqs"] * case["tokens"] * case["q_heads"] * dim * size
        flops += 4.0 * keys * case["tokens"] * case["q_heads"] * dim
    if op == "prompt":
        n = _lengths(case)
        nbytes += sum(n) * 2.0 * (case["q_heads"] + kv) * dim * size
        pairs = sum(x * (x + 1) / 2 if case["causal"] else x * x for x in n)
        flops += 4.0 * pairs * case["q_heads"] * dim
    return {"bytes": nbytes, "flops": flops}
