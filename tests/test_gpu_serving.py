"""The serving operators on the GPU against the float64 oracle: rotary positions and their
gradient, the quantised paged K/V cache, one-token attention, and a decode step of all of them."""
import math

import numpy as np
import pytest
import torch

from gpu_common import fa_module
from oracle import serving as ref

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "s8": torch.int8, "e4m3": torch.float8_e4m3fn}
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}      # half the smallest denormal step


@pytest.fixture(autouse=True)
def _clean_status():
    fa_module().cache_status()
    yield
    fa_module().cache_status()


def np64(t):
    return t.detach().double().cpu().numpy()


def rand(shape, dtype=torch.bfloat16, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- rotary

def check_rotary(x, y, pos, freqs, interleaved, factor, inverse=False):
    want = ref.rotary(np64(x), pos, np64(freqs), interleaved, factor, inverse)
    n, X = freqs.numel(), np.abs(np64(x))
    # One rounding of the result; the angle is off by 2^-24 of half a turn, cos and sin by two
    # units in the last place, products and sum by three roundings: 1e-6 of |x1| + |x2| covers them.
    mate = X.copy()
    one = slice(0, 2 * n, 2) if interleaved else slice(0, n)
    two = slice(1, 2 * n, 2) if interleaved else slice(n, 2 * n)
    mate[..., one], mate[..., two] = X[..., one] + X[..., two], X[..., one] + X[..., two]
    tol = HALF_STEP[x.dtype] * np.abs(want) + 1e-6 * factor * mate + TINY[x.dtype]
    got = np64(y)
    assert np.array_equal(got[..., 2 * n:], np64(x)[..., 2 * n:])
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) / tol).max())


ROTARY = [  # B, HQ, HK, S, D, rot, interleaved, dtype, first position
    (1, 1, 1, 1, 64, 64, False, "bf16", 0), (16, 32, 8, 1, 128, 128, False, "bf16", 1 << 20),
    (2, 3, 1, 33, 128, 64, True, "f16", 7), (1, 4, 2, 300, 64, 24, False, "bf16", 0),
    (2, 5, 5, 17, 96, 26, True, "bf16", 2 ** 31 - 40), (1, 2, 2, 65, 8, 2, False, "f16", 3),
    (1, 2, 1, 129, 192, 192, True, "bf16", 100000), (3, 1, 1, 70, 256, 32, False, "f16", -64),
    (1, 1, 1, 3, 1024, 1024, False, "bf16", 12345), (1, 1, 1, 2, 1024, 1022, True, "f16", 5),
    (1, 16, 16, 1000, 64, 64, False, "bf16", 0), (7, 3, 2, 5, 16, 16, False, "bf16", 9),
    (1, 2, 1, 40, 40, 16, False, "bf16", 9), (2, 3, 1, 50, 192, 24, False, "f16", 9), (1, 2, 2, 9, 1024, 8, False, "bf16", 1),
    (1, 3, 2, 77, 64, 26, False, "bf16", 50), (1, 1, 1, 20, 128, 120, False, "f16", 3), (2, 2, 0, 21, 64, 48, True, "bf16", 9),
]


@pytest.mark.parametrize("case", ROTARY, ids=str)
@pytest.mark.parametrize("inverse", [False, True])
def test_rotary(case, inverse):
    fa = fa_module()
    B, HQ, HK, S, D, rot, inter, dt, first = case
    q, k = rand((B, HQ, S, D), TYPES[dt], 1), rand((B, HK, S, D), TYPES[dt], 2) if HK else None
    pos = (torch.arange(S, device="cuda")[None] + first - 3 * torch.arange(B, device="cuda")[:, None]).to(torch.int32)
    f = fa.rotary_frequencies(rot)
    call = fa.rotary_backward if inverse else fa.rotary
    qo, ko = call(q, k, pos, f, interleaved=inter, factor=1.25)
    for x, y in ((q, qo), (k, ko)):
        if x is not None:
            check_rotary(x, y, np64(pos), f, inter, 1.25, inverse)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", [128, 72])
def test_rotary_strides_positions_and_in_place(inter, rot):
    fa = fa_module()
    f = fa.rotary_frequencies(rot, scaling=fa.FA_ROTARY_SCALE_BY_PARTS, factor=4.0, original_len=1000)
    # (B, S, H, D) memory with a gap between tokens, one row of positions for all sequences
    base = rand((2, 37, 9, 128), seed=3)
    q, k = base[:, :, :6].transpose(1, 2), base[:, :, 6:8].transpose(1, 2)
    pos = torch.randperm(5000, device="cuda")[:37].to(torch.int32)
    rest = base[:, :, 8].clone()
    want_q, want_k = fa.rotary(q.contiguous(), k.contiguous(), pos[None].expand(2, 37).contiguous(), f, interleaved=inter)
    check_rotary(q, want_q, np.tile(np64(pos), (2, 1)), f, inter, 1.0)
    q0, k0 = fa.rotary(q, k, pos, f, interleaved=inter)
    assert torch.equal(q0, want_q) and torch.equal(k0, want_k)
    a, b = fa.rotary(q, k, pos, f, interleaved=inter, q_out=q, k_out=k)
    assert a is q and torch.equal(q, want_q) and torch.equal(k, want_k) and torch.equal(base[:, :, 8], rest)
    x = rand((1, 2, 4, 128), seed=4)
    got, none = fa.rotary(x, None, 11, f, interleaved=inter)
    assert none is None and torch.equal(got, fa.rotary(x, None, i32(11, 12, 13, 14), f, interleaved=inter)[0])


@pytest.mark.parametrize("inter", [False, True])
def test_rotary_gradient_is_the_adjoint(inter):
    # <g, R x> = <R^T g, x> for the kernels' own outputs: each side is off by the rounding of
    # its products alone, half a step of every term.  And R is linear: differences are exact.
    fa = fa_module()
    f = fa.rotary_frequencies(64)
    x, g = rand((2, 3, 50, 128), torch.float16, 5), rand((2, 3, 50, 128), torch.float16, 6)
    pos = torch.arange(50, device="cuda", dtype=torch.int32) * 1000
    y, gx = fa.rotary(x, None, pos, f, interleaved=inter)[0], fa.rotary_backward(g, None, pos, f, interleaved=inter)[0]
    left, right = (g.double() * y.double()).sum(), (gx.double() * x.double()).sum()
    slack = 2.0 ** -11 * ((g.double() * y.double()).abs().sum() + (gx.double() * x.double()).abs().sum())
    assert abs(left - right) <= slack + 1e-5 * slack
    # a step of one element moves the outputs by the step times the gradient's column
    step = torch.zeros_like(x)
    step[1, 2, 17, 5] = 4.0
    col = fa.rotary(step, None, pos, f, interleaved=inter)[0]
    for at in torch.nonzero(col[1, 2, 17]).flatten().tolist():
        one = torch.zeros_like(x)
        one[1, 2, 17, at] = 4.0
        back = fa.rotary_backward(one, None, pos, f, interleaved=inter)[0]
        a, b = float(back[1, 2, 17, 5]), float(col[1, 2, 17, at])
        assert abs(a - b) <= 2 * 2.0 ** -11 * abs(b) + 1e-5


def test_rotary_refusals():
    fa = fa_module()
    q, f = rand((1, 2, 4, 64)), fa.rotary_frequencies(64)
    for bad in (dict(positions=torch.zeros(1, 4, device="cuda")), dict(positions=i32(0, 1, 2)),
                dict(frequencies=f.float()), dict(frequencies=f.cpu()), dict(q=q.cpu()), dict(k=q.cpu())):
        with pytest.raises(ValueError):
            fa.rotary(**{"q": q, "k": None, "positions": i32(0, 1, 2, 3), "frequencies": f, **bad})
    with pytest.raises(ValueError):
        fa.rotary(q, None, 0, f, k_out=q)
    for bad in (q.float(), rand((1, 2, 4, 68))[..., :64]):
        with pytest.raises((TypeError, fa.FaError)):
            fa.rotary(bad, None, 0, f)
    with pytest.raises(fa.FaError):
        fa.rotary(q, None, 0, fa.rotary_frequencies(66))
    e = torch.empty(0, 2, 4, 64, device="cuda", dtype=torch.bfloat16)
    assert fa.rotary(e, None, 0, f)[0].shape == e.shape


# ---------------------------------------------------------------- the cache

def make_cache(kind, n_pages, H, page, D, transposed=False, fill=None):
    fa = fa_module()
    dt = TYPES[kind]
    shape = (n_pages, page, H, D) if transposed else (n_pages, H, page, D)
    pools = []
    for _ in range(2):
        t = torch.zeros(shape, dtype=torch.uint8 if dt.itemsize == 1 else dt, device="cuda")
        if fill is not None:
            t.fill_(fill)
        t = t.view(dt)
        pools.append(t.transpose(1, 2) if transposed else t)
    if dt.itemsize == 1:
        s = [torch.full(shape[:3], -1.0, device="cuda") for _ in range(2)]
        return fa.PagedKVCache(*pools, *[t.transpose(1, 2) if transposed else t for t in s])
    return fa.PagedKVCache(*pools)


def raw(t):
    return t.contiguous().view(torch.uint8) if t.dtype.itemsize == 1 else t.contiguous().view(torch.int16)


def quantised(rows, kind):
    """Codes' values and scales the oracle gives rows (..., D)."""
    return ref.quantise_s8(np64(rows)) if kind == "s8" else ref.quantise_e4m3(np64(rows))


def scattered_table(lens, page, n_pages, seed=0, extra=0):
    """Pages in a random order; entries no sequence needs hold indices outside the pool."""
    rng = np.random.default_rng(seed)
    need = [-(-int(n) // page) for n in lens]
    pages = iter(rng.permutation(n_pages)[:sum(need)])
    width = max(need + [1]) + extra
    t = np.full((len(lens), width), -5, dtype=np.int32)
    t[:, -1] = 2 ** 30
    for b, n in enumerate(need):
        t[b, :n] = [next(pages) for _ in range(n)]
    return torch.from_numpy(t).cuda()


CACHE = [("s8", "bf16", 128, 64), ("s8", "f16", 64, 16), ("e4m3", "bf16", 64, 128), ("e4m3", "f16", 128, 32),
         ("bf16", "bf16", 128, 16), ("f16", "f16", 64, 256)]


@pytest.mark.parametrize("kind, dt, D, page", CACHE)
@pytest.mark.parametrize("transposed", [False, True])
def test_append_and_read(kind, dt, D, page, transposed):
    fa = fa_module()
    H, S, B = 3, 77, 5
    start, count = [0, 5, page - 1, 3 * page + 1, 40], [77, 0, 1, 76, 33]
    end = [s + c for s, c in zip(start, count)]
    n_pages = sum(-(-n // page) for n in end) + 4
    table = scattered_table(end, page, n_pages)
    cache = make_cache(kind, n_pages, H, page, D, transposed, fill=3)
    before = [raw(t).clone() for t in (cache.k, cache.v)]
    x = [rand((B, S, H, D), TYPES[dt], 7 + i, 3.0).transpose(1, 2) for i in range(2)]
    for t in x:                      # rows of every magnitude, and rows whose values tie
        t[0, 0, 3] = 0.0
        t[0, 1, 4] *= 2.0 ** -100 if dt == "bf16" else 2.0 ** -14
        t[0, 2, 5] *= 1e30 if dt == "bf16" else 1e3
        t[0, 0, 6] = torch.linspace(-1, 1, D, device="cuda").to(t.dtype)
        t[0, 1, 7] = (torch.arange(D, device="cuda") % 2 - 0.5).to(t.dtype)      # half of the maximum
        t[0, 1, 7, 0] = 1.0
        for b in range(B):
            t[b, :, count[b]:] = math.nan                # padded rows are not read
    fa.cache_append(cache, *x, table, i32(*start), count=i32(*count))
    out = fa.cache_read(cache, table, i32(*end), S, start=i32(*start), dtype=TYPES[dt])
    assert fa.cache_status() == fa.FA_OK
    touched = np.zeros((n_pages, page), dtype=bool)
    for pool, scales, rows, got in ((cache.k, cache.k_scale, x[0], out[0]), (cache.v, cache.v_scale, x[1], out[1])):
        for b in range(B):
            n = count[b]
            assert not got[b, :, n:].any()               # past the length: zeros
            if n == 0:
                continue
            at = np.arange(start[b], end[b])
            pg, rw = table[b].cpu().numpy()[at // page], at % page
            touched[pg, rw] = True
            mine = pool.view(torch.uint8)[pg, :, rw].view(pool.dtype) if pool.dtype.itemsize == 1 else pool[pg, :, rw]
            mine = mine.transpose(0, 1)                  # (H, n, D)
            if scales is None:
                assert torch.equal(mine, rows[b, :, :n]) and torch.equal(got[b, :, :n], rows[b, :, :n])
                continue
            v, s = quantised(rows[b, :, :n], kind)
            assert np.array_equal(np64(mine), v)         # codes and scales are exact
            assert np.array_equal(np64(scales[pg, :, rw].transpose(0, 1)), s)
            want = v * s[..., None]
            # the product is rounded to fp32 and then once more
            tol = HALF_STEP[TYPES[dt]] * (1 + 2.0 ** -10) * np.abs(want) + TINY[TYPES[dt]]
            assert (np.abs(np64(got[b, :, :n]) - want) <= tol).all()
    for pool, old in ((cache.k, before[0]), (cache.v, before[1])):
        now = raw(pool)
        still = torch.from_numpy(~touched).cuda()
        assert torch.equal(now.transpose(1, 2)[still], old.transpose(1, 2)[still])   # nothing else was written


@pytest.mark.parametrize("kind", ["s8", "e4m3"])
def test_s8_and_e4m3_codes_over_many_rows(kind):
    # 16-bit values meet the borders between codes often; every code has to be the exact one.
    fa = fa_module()
    for dt in ("f16", "bf16"):
        g = torch.Generator(device="cuda").manual_seed(3)
        x = (torch.randint(-127, 128, (1, 1, 8192, 64), generator=g, device="cuda") / 2.0).to(TYPES[dt])
        x[0, 0, :, 0] = (63.5 + torch.arange(8192, device="cuda") / 16.0).to(TYPES[dt])
        cache = make_cache(kind, 64, 1, 128, 64)
        table = torch.arange(64, dtype=torch.int32, device="cuda")[None]
        fa.cache_append(cache, x, x, table, i32(0))
        v, s = quantised(x[0, 0], kind)
        assert np.array_equal(np64(cache.k.reshape(8192, 64)), v)
        assert np.array_equal(np64(cache.v_scale.reshape(8192)), s)


@pytest.mark.parametrize("kind", ["s8", "e4m3", "bf16"])
def test_rows_with_nan_or_infinity(kind):
    fa = fa_module()
    x = rand((1, 2, 6, 64))
    x[0, 0, 1, 3], x[0, 1, 2, 63], x[0, 0, 4, 0] = math.nan, math.inf, -math.inf
    cache = make_cache(kind, 2, 2, 16, 64, fill=1)
    fa.cache_append(cache, x, x, i32(1)[None], i32(2))
    k, _ = fa.cache_read(cache, i32(1)[None], i32(8), 6, start=i32(2))
    if kind == "bf16":
        assert torch.equal(raw(k), raw(x))
    else:
        bad = (~torch.isfinite(x)).any(-1)
        assert torch.isnan(k[bad]).all() and torch.isfinite(k[~bad]).all()
        assert not raw(cache.k[1, :, 2:8])[bad[0]].any()


def test_cache_bad_pages_positions_and_lengths_are_recorded():
    fa = fa_module()
    cache = make_cache("s8", 4, 2, 16, 64, fill=9)
    x = rand((3, 2, 20, 64))
    table = torch.tensor([[0, 1], [2, 4], [-1, 3]], dtype=torch.int32, device="cuda")
    fa.cache_append(cache, x, x, table, i32(20, 0, 0))   # past the table; page 4 of 4; page -1
    assert fa.cache_status() == fa.FA_ERR_INVALID_ARG and fa.cache_status() == fa.FA_OK
    v, s = quantised(x, "s8")
    assert np.array_equal(np64(cache.k[1, :, 4:]), v[0, :, :12]) and np.array_equal(np64(cache.k[2]), v[1, :, :16])
    assert np.array_equal(np64(cache.k[3, :, :4]), v[2, :, 16:]) and (cache.k[3, :, 4:] == 9).all()
    assert (cache.k[0] == 9).all() and (cache.k[1, :, :4] == 9).all()
    fa.cache_append(cache, x[:1], x[:1], table[:1], i32(-3), count=i32(2))
    assert fa.cache_status() == fa.FA_ERR_INVALID_ARG
    k, _ = fa.cache_read(cache, table, i32(40, 20, 20), 24)
    assert fa.cache_status() == fa.FA_ERR_INVALID_ARG
    assert not k[1, :, 16:].any() and not k[2, :, :16].any()
    fa.cache_append(cache, x, x, table, i32(0, 0, 0), count=i32(-7, 0, 0))
    assert fa.cache_status() == fa.FA_OK
    q = rand((3, 4, 1, 64))
    out, lse = fa.decode_attention(q, cache, table, i32(33, -1, 4))
    assert fa.cache_status() == fa.FA_ERR_INVALID_ARG
    assert torch.isfinite(out).all() and not out[1].any() and not out[2].any() and torch.isneginf(lse[1:]).all()
    good, _ = fa.decode_attention(q[:1], cache, table[:1], i32(32))
    assert torch.equal(out[:1], good) and fa.cache_status() == fa.FA_OK


# ---------------------------------------------------------------- decode

def random_cache(kind, lens, page, H, D, seed=0, transposed=False, garbage=True, scale=1.0):
    """A cache with rows for `lens` tokens of each sequence in scattered pages; every other row
    holds NaN (16-bit), a NaN code (e4m3) or a NaN scale.  Returns (cache, table, K, V float64)."""
    need = sum(-(-n // page) for n in lens)
    cache = make_cache(kind, need + 3, H, page, D, transposed)
    table = scattered_table(lens, page, need + 3, seed, extra=1)
    g = torch.Generator(device="cuda").manual_seed(seed)
    host = table.cpu().numpy()
    live = np.zeros((need + 3, page), dtype=bool)
    for b, n in enumerate(lens):
        at = np.arange(n)
        live[host[b][at // page], at % page] = True
    dead = torch.from_numpy(~live).cuda()[:, None].expand(need + 3, H, page)
    whole = []
    for pool, sc in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        x = torch.randn(pool.shape, generator=g, device="cuda") * scale
        if kind == "s8":
            pool.copy_((x * 40).clamp(-127, 127).round().to(torch.int8))
        elif kind == "e4m3":
            x = (x * 60).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            x[dead if garbage else dead & False] = 0x7F
            pool.view(torch.uint8).copy_(x)
        else:
            x[dead if garbage else dead & False] = math.nan
            pool.copy_(x.to(pool.dtype))
        full = np64(pool.float())
        if sc is not None:
            sc.copy_((0.5 + torch.rand(sc.shape, generator=g, device="cuda")) / (40 if kind == "s8" else 60))
            if garbage:
                sc[dead] = math.nan
            full = full * np64(sc)[..., None]
        whole.append(full)
    rows = []
    for full in whole:
        rows.append([full[host[b][np.arange(n) // page], :, np.arange(n) % page].transpose(1, 0, 2) for b, n in enumerate(lens)])
    return cache, table, rows[0], rows[1]


def check_decode(q, out, lse, K, V, lens, window=0, softcap=None, slopes=None, scale=None, kind="bf16", vscale=None):
    # The weights are rounded before their product with V: over an 8-bit cache to fp16 (2^-11), over
    # a 16-bit one to a number of its type and another of the rest (the square of its half step);
    # scores are fp32 sums of D products, the result is rounded once.  fp16 weights
    # (p times the value's scale, the largest at least 1) below 2^-14 are off by up to 2^-25
    # whatever their size: 2^-25 max(p s) |v| / s of each key.
    step = 2.0 ** -11 if kind in ("s8", "e4m3") else HALF_STEP[TYPES[kind]] ** 2
    D = q.shape[3]
    for b, n in enumerate(lens):
        o, l, weight, reach, fine = ref.decode(np64(q[b, :, 0]), K[b], V[b], n, window, softcap, slopes, scale, vscale)
        score = D * 2.0 ** -24 * reach + 2e-6 * (1 + reach)          # a score's error
        if slopes is not None:
            score += 2.0 ** -23 * float(np.abs(slopes).max()) * max(n, 1) * 2
        tol = HALF_STEP[q.dtype] * np.abs(o) + (step + 2 * score + 1e-5) * weight + TINY[q.dtype]
        if kind != "bf16":
            tol += 2.0 ** -25 * fine
        got = np64(out[b, :, 0])
        assert (np.abs(got - o) <= tol).all(), (b, n, float((np.abs(got - o) / tol).max()))
        if lse is not None:
            gl = np64(lse[b, :, 0])
            fin = np.isfinite(l)
            assert np.array_equal(np.isneginf(gl), ~fin)
            assert (np.abs(gl[fin] - l[fin]) <= score + 1e-5 + 2.0 ** -22 * np.abs(l[fin])).all(), (b, n)


RAGGED = [0, 1, 15, 16, 17, 63, 64, 65, 127, 129, 300, 1023, 2049]
DECODE = [  # cache, q dtype, D, kv heads, group, page
    ("bf16", "bf16", 128, 2, 1, 128), ("f16", "f16", 64, 3, 1, 16), ("s8", "bf16", 128, 2, 4, 64),
    ("e4m3", "bf16", 128, 1, 8, 32), ("s8", "f16", 64, 2, 7, 256), ("e4m3", "f16", 64, 1, 12, 16),
    ("bf16", "bf16", 64, 1, 16, 1024), ("f16", "f16", 128, 1, 20, 64), ("s8", "bf16", 128, 1, 33, 16),
    ("e4m3", "bf16", 64, 4, 2, 128), ("bf16", "bf16", 128, 4, 8, 16), ("s8", "f16", 128, 8, 5, 128),
]


@pytest.mark.parametrize("case", DECODE, ids=str)
@pytest.mark.parametrize("window", [0, 1, 100])
def test_decode(case, window):
    fa = fa_module()
    kind, dt, D, H, G, page = case
    cache, table, K, V = random_cache(kind, RAGGED, page, H, D, seed=G, transposed=G % 2 == 1)
    q = rand((len(RAGGED), H * G, 1, D), TYPES[dt], 9, 1.5)
    out, lse = fa.decode_attention(q, cache, table, i32(*RAGGED), window=window)
    assert fa.cache_status() == fa.FA_OK
    check_decode(q, out, lse, K, V, RAGGED, window, kind=kind)
    again, lse2 = fa.decode_attention(q, cache, table, i32(*RAGGED), window=window)
    assert torch.equal(raw(again), raw(out)) and torch.equal(lse, lse2)          # the same bits


@pytest.mark.parametrize("kind", ["bf16", "f16", "s8", "e4m3"])
@pytest.mark.parametrize("B, group, top", [(1, 3, 512), (5, 16, 500), (60, 5, 1024), (3, 2, 1024), (40, 20, 900)])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_over_small_tables(kind, B, group, top, D):
    # Tables that map few tokens: a CTA takes a head's keys alone, or (few heads) they are split.
    fa = fa_module()
    lens = [(top - 17 * b) % (top + 1) for b in range(B)]
    if B > 2:
        lens[1], lens[2] = 0, 1
    cache, table, K, V = random_cache(kind, lens, 32, 3, D, seed=B)
    table = table[:, :-1].contiguous()
    q = rand((B, 3 * group, 1, D), TYPES["f16" if kind == "f16" else "bf16"], 4, 1.5)
    for window in (0, 40):
        out, lse = fa.decode_attention(q, cache, table, i32(*lens), window=window)
        check_decode(q, out, lse, K, V, lens, window, kind=kind)
    assert fa.cache_status() == fa.FA_OK


@pytest.mark.parametrize("kind", ["bf16", "s8"])
@pytest.mark.parametrize("mod", [1, 2, 3])
@pytest.mark.parametrize("window", [0, 70])
def test_decode_score_mods(kind, mod, window):
    fa = fa_module()
    lens = [0, 1, 33, 500, 1500]
    cache, table, K, V = random_cache(kind, lens, 32, 2, 64, seed=mod, scale=2.0)
    q = rand((5, 6, 1, 64), torch.bfloat16, 3, 3.0)
    own = torch.tensor([0.5, 0.25, 0.0, 0.01, 1.0, 0.125], device="cuda")
    for slopes in (None, own):
        s64 = (2.0 ** (-8.0 * np.arange(1, 7) / 6) if slopes is None else np64(own)) if mod & 2 else None
        out, lse = fa.decode_attention(q, cache, table, i32(*lens), window=window, score_mod=mod, softcap=20.0,
                                       alibi_slopes=slopes, scale=0.2)
        check_decode(q, out, lse, K, V, lens, window, 20.0 if mod & 1 else None, s64, 0.2, kind)


@pytest.mark.parametrize("cap", [1e-41, 1e-3, 4.0, 3e3, 1e6, math.inf])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_decode_soft_caps_of_any_size(kind, cap):
    # A cap far above the scores changes nothing (an infinite one: at all); one far below leaves signs.
    fa = fa_module()
    lens = [1, 40, 700]
    cache, table, K, V = random_cache(kind, lens, 32, 2, 64, seed=5, scale=2.0)
    q = rand((3, 6, 1, 64), torch.bfloat16, 3, 3.0)
    out, lse = fa.decode_attention(q, cache, table, i32(*lens), score_mod=fa.FA_SCORE_SOFTCAP, softcap=cap, scale=0.2)
    check_decode(q, out, lse, K, V, lens, softcap=None if math.isinf(cap) else cap, scale=0.2, kind=kind)


@pytest.mark.parametrize("B, HQ, H, n, long", [(40, 64, 4, 60, 9000), (300, 12, 1, 40, 0), (3, 96, 2, 700, 0), (30, 2, 2, 30, 20000),
                                                  (2, 1024, 1, 500, 0)])
def test_decode_many_heads_and_one_long_sequence(B, HQ, H, n, long):
    # The ways in which the parts of a head are joined: heads of no, one, few and very many parts.
    fa = fa_module()
    lens = [(7 * b) % (n + 1) for b in range(B)]
    lens[B // 2] = long or n
    cache, table, K, V = random_cache("s8", lens, 16, H, 64, seed=B)
    q = rand((B, HQ, 1, 64), seed=7, scale=1.5)
    out, lse = fa.decode_attention(q, cache, table, i32(*lens))
    check_decode(q, out, lse, K, V, lens, kind="s8")


@pytest.mark.parametrize("kind, B, HQ, H, n", [("s8", 1, 8, 8, 70001), ("bf16", 1, 32, 2, 40003), ("e4m3", 300, 4, 1, 90),
                                               ("f16", 3, 5, 5, 9000), ("bf16", 700, 2, 2, 1)])
def test_decode_long_contexts_and_large_batches(kind, B, HQ, H, n):
    fa = fa_module()
    lens = [max(0, n - 37 * (b % 9)) for b in range(B)]
    cache, table, K, V = random_cache(kind, lens, 64, H, 128, seed=5)
    q = rand((B, HQ, 1, 128), torch.float16 if kind == "f16" else torch.bfloat16, 2, 2.0)
    out, lse = fa.decode_attention(q, cache, table, i32(*lens))
    check_decode(q, out, lse, K, V, lens, kind=kind)


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("kind", ["bf16", "f16", "s8", "e4m3"])
def test_decode_rows_of_very_different_size(kind, seed):
    # Scales over many orders, a key that takes all the weight late in the sequence, large and
    # tiny queries.
    fa = fa_module()
    torch.manual_seed(seed)
    lens = [900]
    cache, table, K, V = random_cache(kind, lens, 16, 1, 64, seed=1 + seed, garbage=False)
    vs = None
    if cache.quantised:
        f = torch.exp2(torch.randint(-20, 4, cache.v_scale.shape, device="cuda").float())
        cache.v_scale.mul_(f)
        at = torch.arange(900, device="cuda")
        vs = np64(cache.v_scale[table[0].long()[at // 16], :, at % 16]).T
    else:
        cache.k[table[0, 50].item(), 0, 3] *= 30
    K, V = ([gather64(cache, table, 0, 900, w)] for w in (0, 1))
    q = rand((1, 4, 1, 64), torch.float16 if kind == "f16" else torch.bfloat16, 4 + seed)
    q[0, 1] *= 12
    q[0, 2] *= 2.0 ** -12 if kind == "f16" else 2.0 ** -60
    q[0, 3] = 0
    out, lse = fa.decode_attention(q, cache, table, i32(900))
    check_decode(q, out, lse, K, V, lens, kind=kind, vscale=vs)


@pytest.mark.parametrize("kind", ["s8", "e4m3"])
def test_decode_zero_and_tiny_value_rows(kind):
    # Rows of zeros are stored with scale 2^-126: all of them, and a few among others.
    fa = fa_module()
    cache = make_cache(kind, 10, 1, 16, 64)
    table = torch.arange(10, dtype=torch.int32, device="cuda")[None]
    k, v = rand((1, 1, 150, 64), seed=1), torch.zeros(1, 1, 150, 64, dtype=torch.bfloat16, device="cuda")
    q = rand((1, 2, 1, 64), seed=2, scale=2.0)
    for live in ([], [3, 70], [149]):
        v[:, :, live] = rand((1, 1, len(live), 64), seed=3)
        fa.cache_append(cache, k, v, table, i32(0))
        for tiny in (1.0, 2.0 ** -70):
            cache.v_scale.mul_(tiny)
            out, lse = fa.decode_attention(q, cache, table, i32(150))
            at = torch.arange(150, device="cuda")
            vs = np64(cache.v_scale[table[0].long()[at // 16], :, at % 16]).T
            assert torch.isfinite(lse).all()
            check_decode(q, out, lse, [gather64(cache, table, 0, 150, 0)], [gather64(cache, table, 0, 150, 1)], [150],
                         kind=kind, vscale=np.maximum(vs, 2.0 ** -90))


def gather64(cache, table, b, n, which):
    pool, sc = ((cache.k, cache.k_scale), (cache.v, cache.v_scale))[which]
    at = torch.arange(n, device="cuda")
    pg, rw = table[b].long()[at // cache.page_size], at % cache.page_size
    x = pool.view(torch.uint8)[pg, :, rw].view(pool.dtype) if pool.dtype.itemsize == 1 else pool[pg, :, rw]
    x = x.double()
    if sc is not None:
        x = x * sc[pg, :, rw].double()[..., None]
    return np64(x.transpose(0, 1))


@pytest.mark.parametrize("kind", ["bf16", "s8", "e4m3"])
def test_decode_nan_in_a_live_row_stays_in_its_head(kind):
    fa = fa_module()
    cache, table, K, V = random_cache(kind, [200, 200], 32, 2, 64, seed=2, garbage=False)
    q = rand((2, 4, 1, 64), seed=3)
    clean, _ = fa.decode_attention(q, cache, table, i32(200, 200))
    page, row = table[1, 3].item(), 7
    if cache.quantised:
        cache.k_scale[page, 1, row] = math.nan
    else:
        cache.v[page, 1, row, 5] = math.nan
    out, _ = fa.decode_attention(q, cache, table, i32(200, 200))
    assert torch.isnan(out[1, 2:, 0, 5]).all()
    assert torch.equal(out[0], clean[0]) and torch.equal(out[1, :2], clean[1, :2])
    out, _ = fa.decode_attention(q, cache, table, i32(200, 103))                 # now it is not attended to
    assert torch.isfinite(out).all()


def test_decode_beyond_32_bit_offsets():
    fa = fa_module()
    H, page, D, n = 8, 128, 128, 200
    n_pages = 2 ** 31 // (H * page * D) + 40                                     # elements past 2^31
    for kind in ("s8", "bf16"):
        k, v = (torch.empty(n_pages, H, page, D, dtype=TYPES[kind], device="cuda") for _ in range(2))
        sc = [torch.empty(n_pages, H, page, device="cuda") for _ in range(2)] if kind == "s8" else []
        cache = fa.PagedKVCache(k, v, *sc)
        table = i32(n_pages - 1, n_pages - 2)[None]
        x = [rand((1, H, n, D), seed=i) for i in range(2)]
        fa.cache_append(cache, *x, table, i32(0))
        K, V = fa.cache_read(cache, table, i32(n), n)
        tol = 0 if kind == "bf16" else 2.0 ** -8 + 0.51 / 127
        for a, b in ((K, x[0]), (V, x[1])):
            assert ((a.double() - b.double()).abs() <= tol * b.double().abs().amax(-1, keepdim=True)).all()
        q = rand((1, 16, 1, D), seed=5)
        out, lse = fa.decode_attention(q, cache, table, i32(n))
        check_decode(q, out, lse, [gather64(cache, table, 0, n, 0)], [gather64(cache, table, 0, n, 1)], [n], kind=kind)
        del k, v, sc, cache
        torch.cuda.empty_cache()


def test_decode_strides_streams_and_own_buffers():
    fa = fa_module()
    lens = [130, 64]
    cache, table, K, V = random_cache("e4m3", lens, 16, 2, 128, seed=8)
    wide = torch.full((2, table.shape[1] + 5), 7, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    q = rand((2, 1, 8, 128), seed=1).transpose(1, 2)                             # (B, 1, HQ, D) memory
    base, blse = fa.decode_attention(q.contiguous(), cache, table, i32(*lens))
    out = torch.full((2, 8, 2, 128), 5.0, dtype=torch.bfloat16, device="cuda")[:, :, :1]
    lse = torch.empty(2, 8, 1, device="cuda")
    ws = torch.empty(fa.decode_workspace_bytes(2, 8, 2, 128) + 16, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got, none = fa.decode_attention(q, cache, wide[:, :table.shape[1]], i32(*lens), out=out, lse=lse, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    assert got is out and torch.equal(out, base) and torch.equal(lse, blse)
    assert (out.as_strided((2, 8, 128), (2048, 256, 1), 128) == 5).all()         # the gap rows
    check_decode(q, out, lse, K, V, lens, kind="e4m3")
    assert fa.decode_attention(q, cache, table, i32(*lens), return_lse=False)[1] is None
    for s in (side, side.cuda_stream):                   # the stream as an argument
        side.wait_stream(torch.cuda.current_stream())
        got, glse = fa.decode_attention(q, cache, table, i32(*lens), stream=s)
        torch.cuda.synchronize()
        assert torch.equal(got, base) and torch.equal(glse, blse)
    with pytest.raises(fa.FaError, match="workspace"):
        fa.decode_attention(q, cache, table, i32(*lens), workspace=ws[:8])


def test_decode_refusals():
    fa = fa_module()
    cache, table, _, _ = random_cache("s8", [20, 20], 16, 2, 64)
    q, n = rand((2, 4, 1, 64)), i32(20, 20)
    for bad in (dict(q=q.cpu()), dict(kv_lens=n.long()), dict(kv_lens=n[:1]), dict(kv_lens=n.cpu()),
                dict(page_table=table[:1]), dict(page_table=table.long()), dict(lse=torch.empty(2, 4, device="cuda")),
                dict(out=q.cpu()), dict(window=2 ** 32 + 5), dict(workspace=torch.empty(1 << 24, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            fa.decode_attention(**{"q": q, "cache": cache, "page_table": table, "kv_lens": n, **bad})
    for bad in (rand((2, 3, 1, 64)), rand((2, 4, 2, 64)), rand((2, 4, 1, 128))):
        with pytest.raises(fa.FaError):
            fa.decode_attention(bad, cache, table, n)
    with pytest.raises(fa.FaError):
        fa.decode_attention(q, cache, table, n, score_mod=fa.FA_SCORE_SOFTCAP, softcap=0.0)
    with pytest.raises(ValueError):
        fa.PagedKVCache(cache.k, cache.v)
    with pytest.raises(ValueError):
        fa.PagedKVCache(cache.k, cache.v[:1], cache.k_scale, cache.v_scale)
    with pytest.raises(fa.FaError):
        c = fa.PagedKVCache.empty(2, 2, 24, 64, torch.bfloat16)
        fa.decode_attention(q, c, table, n)
    with pytest.raises(fa.FaError):
        fa.cache_append(make_cache("f16", 2, 2, 16, 64), q[:, :2], q[:, :2], table, i32(0, 0))
    with pytest.raises(TypeError):
        fa.cache_read(cache, table, n, 4, dtype=torch.float32)
    with pytest.raises(ValueError):
        fa.cache_read(cache, table, n, -1)
    with pytest.raises(ValueError):
        fa.cache_append(cache, q[:, :2], q[:, :2].cpu(), table, i32(0, 0))
    with pytest.raises(ValueError):
        fa.cache_append(cache, q[:, :2], q[:, :2], table, i32(0, 0), count=i32(1))
    with pytest.raises(ValueError):
        fa.cache_read(cache, table, n, 4, k_out=torch.empty(2, 2, 5, 64, dtype=torch.bfloat16, device="cuda"))
    none = torch.empty(0, 4, 1, 64, dtype=torch.bfloat16, device="cuda")
    assert fa.decode_attention(none, cache, table[:0], n[:0])[0].shape == none.shape


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("kind", ["s8", "bf16"])
def test_a_prompt_and_captured_decode_steps(kind):
    """A prompt goes through rotary, fa_forward and the cache; then a decode step, captured once,
    is replayed while lengths, positions and tokens change in device memory."""
    fa = fa_module()
    B, HQ, H, D, page, S, steps = 2, 8, 2, 64, 16, 61, 5
    f = fa.rotary_frequencies(D)
    lens = [61, 40]
    cache = make_cache(kind, 20, H, page, D, fill=1)
    table = scattered_table([S + steps] * B, page, 20, 3)
    k, v = rand((B, H, S, D), seed=1), rand((B, H, S, D), seed=2)
    q, kr = fa.rotary(rand((B, HQ, S, D), seed=3), k, 0, f)
    fa.cache_append(cache, kr, v, table, i32(0, 0), count=i32(*lens))
    kc, vc = fa.cache_read(cache, table, i32(*lens), S)
    bm = fa.create_block_mask(fa.FA_MASK_CAUSAL, B, None, S, S, kv_lens=i32(*lens))
    out, _ = fa.flex_attention(q, kc.repeat_interleave(HQ // H, 1), vc.repeat_interleave(HQ // H, 1), bm)
    for b in range(B):                                   # the prompt's last token, both ways
        n = lens[b]
        one, _ = fa.decode_attention(q[b:b + 1, :, n - 1:n].contiguous(), cache, table[b:b + 1], i32(n))
        assert (one.double() - out[b:b + 1, :, n - 1:n].double()).abs().max() <= 2e-2
    # static buffers of the captured step
    tq, tk, tv = (torch.zeros(B, h, 1, D, dtype=torch.bfloat16, device="cuda") for h in (HQ, H, H))
    pos, now = i32(0, 0)[:, None], i32(1, 1)
    ws = torch.empty(fa.decode_workspace_bytes(B, HQ, H, D), dtype=torch.uint8, device="cuda")
    res, rl = torch.zeros_like(tq), torch.zeros(B, HQ, 1, device="cuda")

    def step():
        a, c = fa.rotary(tq, tk, pos, f)
        fa.cache_append(cache, c, tv, table, pos[:, 0])
        fa.decode_attention(a, cache, table, now, out=res, lse=rl, workspace=ws)
        return a

    pos[:, 0] = i32(*lens)
    now.copy_(i32(*lens) + 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        turned = step()
    for t in range(steps):
        for buf, s in ((tq, 10), (tk, 20), (tv, 30)):
            buf.copy_(rand(buf.shape, seed=s + t))
        graph.replay()
        torch.cuda.synchronize()
        at = [n + t + 1 for n in lens]
        check_decode(turned, res, rl, *[[gather64(cache, table, b, at[b], w) for b in range(B)] for w in (0, 1)], at, kind=kind)
        pos += 1
        now += 1
    assert fa.cache_status() == fa.FA_OK


def test_two_decodes_at_once():
    fa = fa_module()
    lens = [3000, 10, 777]
    cache, table, K, V = random_cache("s8", lens, 64, 4, 128, seed=6)
    qs = [rand((3, 16, 1, 128), seed=s) for s in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for s, q in zip(streams, qs):
            with torch.cuda.stream(s):
                got.append(fa.decode_attention(q, cache, table, i32(*lens)))
    torch.cuda.synchronize()
    for i, (out, lse) in enumerate(got):
        check_decode(qs[i % 2], out, lse, K, V, lens, kind="s8")
