"""Performance cases of the serving operators: rotary positions, the quantised paged K/V cache,
and attention of one new token over that cache.

Each case runs either the operator's plain form (elementary torch operations in 32 bits, 64
where 32 lose what matters) or, with ``own``, the library's entry points on the same inputs.
``exact`` gives the outputs from the operators' definitions in 64 bits.

Definitions shared by the forms below
  rotary      pair (x1, x2) of position t turns by the angle a = t * f_i:
              y1 = c (x1 cos a - x2 sin a), y2 = c (x2 cos a + x1 sin a); the gradient turns by -a
  s8 row      scale = max(fp32(max|x| / 127), 2^-126), code = x / scale rounded to even
  e4m3 row    scale = the smallest power of two >= 2^-126 with max|x| / scale <= 448,
              code = x / scale rounded to even among the e4m3 values
  read back   code * scale; rows past a sequence's length are zero
  decode      softmax over the keys max(0, len - window) <= j < len of
              mod(scale * q.k_j), times v; no key: out 0, lse -inf
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "s8": torch.int8, "e4m3": torch.float8_e4m3fn}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # One decode step of 16 sequences far into their contexts: latency is everything.
        dict(name="rotary_step", op="rotary", B=16, HQ=32, HK=8, S=1, D=128, rot=128, layout="half", dtype="bf16",
             grad=False, parts=False, far=1 << 20),
        # The q and k of the 8k causal training workload (16 heads, D = 64).
        dict(name="rotary_8k", op="rotary", B=1, HQ=16, HK=16, S=8192, D=64, rot=64, layout="half", dtype="bf16",
             grad=False, parts=False, far=0),
        # The gradient at 32k positions: interleaved pairs in half of the head, scaled by parts.
        dict(name="rotary_grad_32k", op="rotary", B=1, HQ=32, HK=8, S=32768, D=128, rot=64, layout="interleaved",
             dtype="f16", grad=True, parts=True, far=0),
        # One new token of 16 sequences written as 8-bit integers and read back.
        dict(name="cache_step_s8", op="cache", B=16, H=8, S=1, D=128, cache="s8", dtype="bf16", page=64, lo=1024,
             hi=8192, append=True),
        # Ragged prompts of up to 8k tokens written in e4m3 (a padded batch) and read back.
        dict(name="cache_prompt_e4m3", op="cache", B=4, H=8, S=8192, D=128, cache="e4m3", dtype="bf16", page=128,
             lo=1000, hi=8192, append=True),
        # The contexts of 16 sequences read back for another prefill over them.
        dict(name="cache_read_s8", op="cache", B=16, H=16, S=8192, D=128, cache="s8", dtype="bf16", page=128, lo=1024,
             hi=8192, append=False),
        # The smallest decode call: one short sequence, one page past a boundary.
        dict(name="decode_short", op="decode", B=1, HQ=8, HK=8, D=64, cache="f16", dtype="f16", page=16, lo=257, hi=257,
             idle=0, window=0, mod="none"),
        # The paged decode workload: 16 sequences x 16 heads, 1k-8k contexts, bf16 pages of 128.
        dict(name="decode_16x16_bf16", op="decode", B=16, HQ=16, HK=16, D=128, cache="bf16", dtype="bf16", page=128,
             lo=1024, hi=8192, idle=0, window=0, mod="none"),
        # The same contexts with grouped heads and an 8-bit cache.
        dict(name="decode_grouped_s8", op="decode", B=16, HQ=64, HK=8, D=128, cache="s8", dtype="bf16", page=64,
             lo=1024, hi=8192, idle=0, window=0, mod="none"),
        # One long context, split over the whole GPU.
        dict(name="decode_128k_e4m3", op="decode", B=1, HQ=32, HK=8, D=128, cache="e4m3", dtype="bf16", page=128,
             lo=131072, hi=131072, idle=0, window=0, mod="none"),
        # A large serving batch with idle slots, soft-capped scores.
        dict(name="decode_batch_bf16", op="decode", B=96, HQ=32, HK=8, D=128, cache="bf16", dtype="bf16", page=16,
             lo=500, hi=16384, idle=5, window=0, mod="softcap"),
        # A whole attention step of a decode: rotary positions, cache write, attention.
        dict(name="step_s8", op="step", B=16, HQ=32, HK=8, D=128, cache="s8", dtype="bf16", page=64, lo=1024, hi=8192,
             idle=0, window=0, mod="none"),
    ]


def _log(rng, a, b):
    return max(a, min(b, int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))))


def draw(rng):
    """One case of the ranges; a very large one gives way to the next."""
    case = _any(rng)
    return case if work(case)["bytes"] <= 1.4e9 else draw(rng)


def _any(rng):
    op = rng.choice(["rotary", "cache", "decode", "decode", "step"])
    D = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "f16"])
    if op == "rotary":
        HK = rng.choice([1, 2, 4, 8, 16])
        S = _log(rng, 1, 32768)
        D = rng.choice([64, 128, 192])
        return dict(op=op, B=rng.randint(1, max(1, min(16, 65536 // S))), HQ=HK * rng.choice([1, 2, 4]), HK=HK, S=S, D=D,
                    rot=rng.choice([D, D // 2, D // 4, 24]), layout=rng.choice(["half", "interleaved"]), dtype=dtype,
                    grad=rng.random() < 0.5, parts=rng.random() < 0.5, far=rng.choice([0, 1 << 17, 1 << 20]))
    cache = rng.choice(["s8", "e4m3", dtype])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "cache":
        S = _log(rng, 1, 16384)
        append = rng.random() < 0.6
        return dict(op=op, B=rng.randint(1, max(1, min(32, 65536 // S))), H=rng.choice([1, 2, 4, 8, 16]), S=S, D=D,
                    cache=cache, dtype=dtype, page=page, lo=max(1, S // 3), hi=S + rng.choice([0, 1, 77]), append=append)
    hi = _log(rng, 1, 65536)
    B = rng.randint(1, max(1, min(128, 400000 // hi)))
    HK = rng.choice([1, 2, 4, 8])
    return dict(op=op, B=B, HQ=HK * rng.choice([1, 2, 4, 5, 7, 8, 12, 16]), HK=HK, D=D, cache=cache, dtype=dtype, page=page,
                lo=max(1, hi // rng.choice([1, 2, 8])), hi=hi, idle=rng.choice([0, 0, B // 4]) if op == "decode" else 0,
                window=rng.choice([0, 0, 1, 333, 4096]), mod=rng.choice(["none", "softcap", "alibi", "both"]))


# ---------------------------------------------------------------- inputs

def _lengths(case):
    """Lengths spread over [lo, hi] in their logarithm, the last `idle` of them zero (their
    order goes by the seed)."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    busy = B - case.get("idle", 0)
    return [int(round(lo * (hi / lo) ** (i / (B - 1) if B > 1 else 1.0))) if i < busy else 0 for i in range(B)]


def _frequencies(rot, parts):
    """Angles a position (radians) of base 10000; by parts: slow pairs divided by 8."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    if parts:
        ramp = ((4096.0 * f / (2 * math.pi) - 1.0) / 31.0).clamp(0.0, 1.0)
        f = f / 8.0 * (1.0 - ramp) + f * ramp
    return f


def _rows(g, shape, dtype):
    """Rows with a few loud channels, as keys and values have them."""
    loud = 1.0 + 7.0 * (torch.rand(shape[-1], generator=g, device="cuda") < 0.05)
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * loud).to(dtype)


def _pool(g, case, H):
    """The pages of a cache in use: codes and scales of 8-bit types, plain rows of 16-bit ones."""
    need = [-(-max(1, n) // case["page"]) for n in _lengths(case)]
    shape = (sum(need) + 3, H, case["page"], case["D"])
    kind = _TYPES[case["cache"]]
    if case["cache"] == "s8":
        made = [torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8) for _ in range(2)]
    else:
        loud = 100.0 if case["cache"] == "e4m3" else 1.0
        made = [(torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16) * loud).clamp(-448, 448).to(kind)
                for _ in range(2)]
    scales = [None, None]
    if case["cache"] in ("s8", "e4m3"):
        unit = 1 / 64 if case["cache"] == "s8" else 1 / 128
        scales = [unit * (0.5 + torch.rand(shape[:3], generator=g, device="cuda")) for _ in range(2)]
    order = torch.randperm(shape[0], generator=g, device="cuda").to(torch.int32)
    lens = torch.tensor(_lengths(case), dtype=torch.int32)
    need = torch.tensor(need)
    at = torch.randperm(case["B"], generator=torch.Generator().manual_seed(g.initial_seed()))
    lens, need = lens[at], need[at]
    first = (torch.cumsum(need, 0) - need).cuda()
    width = int(need.max())
    page = first[:, None] + torch.arange(width, device="cuda").minimum(need.cuda()[:, None] - 1)
    table = order[page].contiguous()
    return made[0], made[1], scales[0], scales[1], table, lens.cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case)
    kind = _TYPES[case["dtype"]]
    if case["op"] in ("rotary", "step"):
        S = case.get("S", 1)
        rot = case.get("rot", case["D"])
        s["q"] = _rows(g, (case["B"], case["HQ"], S, case["D"]), kind)
        s["k"] = _rows(g, (case["B"], case["HK"], S, case["D"]), kind)
        s["f"] = _frequencies(rot, case.get("parts", False))
        s["c"] = 0.1 * math.log(8.0) + 1.0 if case.get("parts") else 1.0
        if case["op"] == "rotary":
            first = torch.randint(0, max(1, case["far"]), (case["B"], 1), generator=g, device="cuda")
            s["pos"] = (first + torch.arange(S, device="cuda")).to(torch.int32)
    if case["op"] == "cache":
        H, S = case["H"], case["S"]
        pool = _pool(g, case, H)
        s["pool"], s["table"], s["lens"] = pool[:4], pool[4], pool[5]
        s["start"] = (s["lens"] - S).clamp_min(0)
        s["count"] = s["lens"] - s["start"]
        if case["append"]:
            s["k"], s["v"] = (_rows(g, (case["B"], H, S, case["D"]), kind) for _ in range(2))
    if case["op"] in ("decode", "step"):
        pool = _pool(g, case, case["HK"])
        s["pool"], s["table"], s["lens"] = pool[:4], pool[4], pool[5]
        if case["op"] == "decode":
            s["q"] = _rows(g, (case["B"], case["HQ"], 1, case["D"]), kind)
        else:
            s["v"] = _rows(g, (case["B"], case["HK"], 1, case["D"]), kind)
            s["start"] = s["lens"] - 1
            s["pos"] = s["start"][:, None].contiguous()
    if own and "pool" in s:
        # The cache's handle, which a serving program makes once for its pools.
        import block_sparse_masked_x128_b200 as fa
        s["cache_handle"] = fa.PagedKVCache(*s["pool"])
    return s


# ---------------------------------------------------------------- the plain forms

def _rotary(x, pos, f, c, layout, sign):
    a = pos.double()[:, None, :, None] * f                                   # (B, 1, S, rot / 2)
    cos, sin = (a.cos() * c).float(), (a.sin() * (c * sign)).float()
    rot = 2 * f.numel()
    r, rest = x[..., :rot].float(), x[..., rot:]
    if layout == "half":
        x1, x2 = r[..., :rot // 2], r[..., rot // 2:]
    else:
        x1, x2 = r[..., 0::2], r[..., 1::2]
    y1, y2 = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    y = torch.cat((y1, y2), -1) if layout == "half" else torch.stack((y1, y2), -1).flatten(-2)
    return torch.cat((y.to(x.dtype), rest), -1)


def _quantise(x, cache):
    """Codes and scales of rows (..., D); the division in 64 bits keeps borders where they are."""
    if cache not in ("s8", "e4m3"):
        return x, None
    amax = x.float().abs().amax(-1)
    if cache == "s8":
        scale = (amax / 127).clamp_min(2.0 ** -126)
        return (x.double() / scale.double()[..., None]).round().to(torch.int8), scale
    m = torch.frexp(amax).mantissa                                           # amax = m 2^e, 1/2 <= m < 1
    scale = torch.where(amax > 0, amax / m * torch.where(m <= 0.875, 2.0 ** -9, 2.0 ** -8), 0.0).clamp_min(2.0 ** -126)
    return (x.float() / scale[..., None]).to(torch.float8_e4m3fn), scale


def _slots(table, pos, page):
    """Page and row of positions (B, S) of their sequences."""
    return table.long().gather(1, (pos // page).clamp(0, table.shape[1] - 1).long()), (pos % page).long()


def _append(pool, x, scale_pool, table, start, count, page, cache):
    B, H, S, D = x.shape
    s = torch.arange(S, device=x.device)
    live = s[None] < count[:, None]
    pages, rows = _slots(table, start[:, None] + s[None], page)
    pages, rows = pages[live], rows[live]
    codes, scale = _quantise(x.transpose(1, 2)[live], cache)                 # (tokens, H, D)
    raw = pool.view(torch.uint8) if cache == "e4m3" else pool
    raw[pages, :, rows] = codes.view(torch.uint8) if cache == "e4m3" else codes
    if scale is not None:
        scale_pool[pages, :, rows] = scale


def _gather(pool, scale_pool, table, pos, page):
    """fp32 rows (B, H, S, D) of positions (B, S)."""
    pages, rows = _slots(table, pos, page)
    x = pool.view(torch.uint8)[pages, :, rows].view(pool.dtype) if pool.dtype == torch.float8_e4m3fn else pool[pages, :, rows]
    x = x.float()
    if scale_pool is not None:
        x = x * scale_pool[pages, :, rows][..., None]
    return x.transpose(1, 2)


def _read(s, dtype):
    pos = s["start"][:, None] + torch.arange(s.get("S", 1), device="cuda")[None]
    live = (pos < s["lens"][:, None])[:, None, :, None]
    k, v, ks, vs = s["pool"]
    return [torch.where(live, _gather(p, c, s["table"], pos, s["page"]), 0.0).to(dtype) for p, c in ((k, ks), (v, vs))]


def _slopes(H):
    return 2.0 ** (-8.0 * torch.arange(1, H + 1, device="cuda", dtype=torch.float32) / H)


def _decode(q, s):
    B, HQ, _, D = q.shape
    HK = s["HK"]
    k, v, ks, vs = s["pool"]
    L = int(s["hi"])
    pos = torch.arange(L, device="cuda")[None].expand(B, L)
    K, V = _gather(k, ks, s["table"], pos, s["page"]), _gather(v, vs, s["table"], pos, s["page"])
    x = torch.matmul(q.float().reshape(B, HK, HQ // HK, D), K.transpose(2, 3)) * (D ** -0.5)
    if s["mod"] in ("softcap", "both"):
        x = 30.0 * torch.tanh(x / 30.0)
    lens = s["lens"][:, None]
    if s["mod"] in ("alibi", "both"):
        x = x + _slopes(HQ).reshape(1, HK, HQ // HK, 1) * (pos - (lens - 1)).float()[:, None, None]
    live = pos < lens
    if s["window"]:
        live = live & (pos >= lens - s["window"])
    x = x.masked_fill(~live[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, 0.0)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    out = torch.where(total > 0, torch.matmul(p, V) / total, 0.0)
    return out.reshape(B, HQ, 1, D).to(q.dtype), (torch.log(total) + m).reshape(B, HQ, 1)


def run(state):
    s = state
    if own:
        return _run_own(s)
    if s["op"] == "rotary":
        sign = -1.0 if s["grad"] else 1.0
        return [_rotary(x, s["pos"], s["f"], s["c"], s["layout"], sign) for x in (s["q"], s["k"])]
    k, v, ks, vs = s["pool"]
    if s["op"] == "cache":
        if s["append"]:
            _append(k, s["k"], ks, s["table"], s["start"], s["count"], s["page"], s["cache"])
            _append(v, s["v"], vs, s["table"], s["start"], s["count"], s["page"], s["cache"])
        return _read(s, _TYPES[s["dtype"]])
    if s["op"] == "decode":
        return list(_decode(s["q"], s))
    q, knew = (_rotary(x, s["pos"], s["f"], s["c"], "half", 1.0) for x in (s["q"], s["k"]))
    one = torch.ones_like(s["start"])
    _append(k, knew, ks, s["table"], s["start"], one, s["page"], s["cache"])
    _append(v, s["v"], vs, s["table"], s["start"], one, s["page"], s["cache"])
    return [_decode(q, s)[0]] + _read(s, q.dtype)


# ---------------------------------------------------------------- the library's calls

def _mod(fa, s):
    return {"none": 0, "softcap": fa.FA_SCORE_SOFTCAP, "alibi": fa.FA_SCORE_ALIBI,
            "both": fa.FA_SCORE_SOFTCAP | fa.FA_SCORE_ALIBI}[s["mod"]]


def _run_own(s):
    import block_sparse_masked_x128_b200 as fa
    if s["op"] == "rotary":
        call = fa.rotary_backward if s["grad"] else fa.rotary
        return list(call(s["q"], s["k"], s["pos"], s["f"], interleaved=s["layout"] == "interleaved", factor=s["c"]))
    cache = s["cache_handle"]
    if s["op"] == "cache":
        if s["append"]:
            fa.cache_append(cache, s["k"], s["v"], s["table"], s["start"], count=s["count"])
        return list(fa.cache_read(cache, s["table"], s["lens"], s["S"], start=s["start"], dtype=_TYPES[s["dtype"]]))
    if s["op"] == "decode":
        return list(fa.decode_attention(s["q"], cache, s["table"], s["lens"], window=s["window"], score_mod=_mod(fa, s)))
    q, k = fa.rotary(s["q"], s["k"], s["pos"], s["f"], factor=s["c"])
    fa.cache_append(cache, k, s["v"], s["table"], s["start"])
    out, _ = fa.decode_attention(q, cache, s["table"], s["lens"], window=s["window"], score_mod=_mod(fa, s), return_lse=False)
    return [out, *fa.cache_read(cache, s["table"], s["lens"], 1, start=s["start"], dtype=q.dtype)]


# ---------------------------------------------------------------- work and the definitions in 64 bits

def work(case):
    D, B = case["D"], case["B"]
    if case["op"] == "rotary":
        n = B * case["S"] * (case["HQ"] + case["HK"])
        return {"bytes": 4 * n * D + 4 * B * case["S"] + 4 * case["rot"], "flops": 3 * n * case["rot"]}
    size = {"s8": 1, "e4m3": 1}.get(case["cache"], 2)
    row = D * size + (4 if size == 1 else 0)                                 # a cached row and its scale
    lens = _lengths(case)
    if case["op"] == "cache":
        rows = 2 * case["H"] * sum(min(n, case["S"]) for n in lens)
        move = rows * row + 2 * case["H"] * B * case["S"] * 2 * D            # read, and the padded result written
        return {"bytes": move + (rows * (2 * D + row) if case["append"] else 0), "flops": rows * D * (3 if case["append"] else 1)}
    keys = sum(min(n, case["window"] or n) for n in lens)
    w = {"bytes": 2 * keys * case["HK"] * row + 4 * B * case["HQ"] * D, "flops": 4 * keys * case["HQ"] * D}
    if case["op"] == "decode":
        w["bytes"] += 4 * B * case["HQ"]                                     # lse
    else:
        w["bytes"] += 4 * B * (case["HQ"] + case["HK"]) * D + 2 * B * case["HK"] * (2 * D + 2 * row + 2 * D)
    return w


def _turned(x, pos, f, c, layout, sign):
    """Rotation as a product of complex numbers in 64 bits."""
    z = torch.polar(torch.full((), float(c), dtype=torch.float64, device="cuda"), sign * pos.double().unsqueeze(-1) * f)
    n = f.numel()
    x = x.double()
    pair = torch.complex(x[..., :n], x[..., n:2 * n]) if layout == "half" else torch.view_as_complex(
        x[..., :2 * n].reshape(*x.shape[:-1], n, 2).contiguous())
    y = pair * z[:, None]
    turned = torch.cat((y.real, y.imag), -1) if layout == "half" else torch.view_as_real(y).flatten(-2)
    return torch.cat((turned, x[..., 2 * n:]), -1)


def _stands_for(x, cache):
    """The values that a row's codes stand for, in 64 bits."""
    x = x.double()
    if cache not in ("s8", "e4m3"):
        return x
    top = x.abs().max(-1, keepdim=True).values
    if cache == "s8":
        scale = (top / 127.0).float().double().clamp_min(2.0 ** -126)
        return torch.round(x / scale) * scale
    scale = torch.exp2(torch.ceil(torch.log2(top.clamp_min(2.0 ** -200) / 448.0)).clamp_min(-126.0))
    scale = torch.where(top > 448.0 * scale, 2 * scale, scale)
    scale = torch.where((top <= 224.0 * scale) & (scale > 2.0 ** -126), scale / 2, scale)
    y = x / scale
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3.0)
    return torch.round(y / step) * step * scale


def _row64(s, n, which):
    """Rows 0..n-1 of sequence n[0] as the cache holds them before the call, in 64 bits: (H, n, D)."""
    b, length = n
    t = torch.arange(length, device="cuda")
    page, row = s["table"][b].long()[t // s["page"]], t % s["page"]
    pool = s["pool"][which]
    x = (pool.view(torch.uint8)[page, :, row].view(pool.dtype) if pool.dtype == torch.float8_e4m3fn else pool[page, :, row]).double()
    if s["pool"][2 + which] is not None:
        x = x * s["pool"][2 + which][page, :, row].double().unsqueeze(-1)
    return x.transpose(0, 1)


def exact(case, seed):
    s = prepare(case, seed)
    sign = -1.0 if case.get("grad") else 1.0
    if case["op"] == "rotary":
        return [_turned(x, s["pos"], s["f"], s["c"], case["layout"], sign) for x in (s["q"], s["k"])]
    lens, start = s["lens"].tolist(), s["start"].tolist() if "start" in s else None
    kind = _TYPES[case["dtype"]]
    if case["op"] == "cache":
        outs = []
        for which, name in ((0, "k"), (1, "v")):
            y = torch.zeros(case["B"], case["H"], case["S"], case["D"], dtype=torch.float64, device="cuda")
            for b in range(case["B"]):
                n = lens[b] - start[b]
                y[b, :, :n] = _stands_for(s[name][b, :, :n], case["cache"]) if case["append"] else _row64(s, (b, lens[b]), which)[:, start[b]:]
            outs.append(y)
        return outs
    q = s["q"].double()
    new = [None, None]
    if case["op"] == "step":
        q = _turned(s["q"], s["pos"], s["f"], s["c"], "half", 1.0).to(kind).double()
        k = _turned(s["k"], s["pos"], s["f"], s["c"], "half", 1.0).to(kind)
        new = [_stands_for(k, case["cache"]), _stands_for(s["v"], case["cache"])]
    HQ, HK, D = case["HQ"], case["HK"], case["D"]
    out = torch.zeros(case["B"], HQ, 1, D, dtype=torch.float64, device="cuda")
    lse = torch.full((case["B"], HQ, 1), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        n = lens[b]
        if n == 0:
            continue
        K, V = _row64(s, (b, n), 0), _row64(s, (b, n), 1)
        if case["op"] == "step":
            K[:, n - 1], V[:, n - 1] = new[0][b, :, 0], new[1][b, :, 0]
        at = max(0, n - case["window"]) if case["window"] else 0
        x = torch.einsum("hgd,hnd->hgn", q[b, :, 0].reshape(HK, HQ // HK, D), K[:, at:]) / math.sqrt(D)
        if case["mod"] in ("softcap", "both"):
            x = 30.0 * torch.tanh(x / 30.0)
        if case["mod"] in ("alibi", "both"):
            slope = torch.exp2(-8.0 * torch.arange(1, HQ + 1, device="cuda", dtype=torch.float64) / HQ)
            x = x + slope.reshape(HK, -1, 1) * torch.arange(at - (n - 1), 1, device="cuda", dtype=torch.float64)
        lse[b, :, 0] = torch.logsumexp(x, -1).flatten()
        out[b, :, 0] = torch.einsum("hgn,hnd->hgd", torch.softmax(x, -1), V[:, at:]).reshape(HQ, D)
    return [out, new[0], new[1]] if case["op"] == "step" else [out, lse]
