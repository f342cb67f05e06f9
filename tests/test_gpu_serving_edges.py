"""The serving operators at the edges of their numbers and arguments: infinities and the largest
values in a cache, row scales over the whole range of fp32, non-finite frequencies."""
import math

import numpy as np
import pytest
import torch

from gpu_common import fa_module
from oracle import serving as ref
from test_gpu_serving import (TYPES, _clean_status, check_decode, check_rotary, gather64, i32, make_cache,  # noqa: F401
                              np64, rand, random_cache, raw)

pytestmark = pytest.mark.gpu

# Lengths whose tables map few tokens (a CTA takes a head alone) and many (the keys are split).
NARROW, WIDE = [1, 17, 40, 300], [1, 17, 40, 3000]
# Split keys again, several steps to a warp.
MANY = [3000 - 7 * b for b in range(90)]


def rows64(cache, table, lens):
    """The cached K and V of each sequence, (H, n, D) float64."""
    return [[gather64(cache, table, b, n, w) for b, n in enumerate(lens)] for w in (0, 1)]


def put(cache, table, b, key, head, dim, value):
    cache.v[table[b, key // cache.page_size].item(), head, key % cache.page_size, dim] = value


# ---------------------------------------------------------------- workspaces

def test_decode_refuses_a_workspace_that_is_not_contiguous():
    # A broadcast or strided tensor's size in bytes is more than the memory behind it.
    fa = fa_module()
    cache, table, _, _ = random_cache("s8", [20, 20], 16, 2, 64)
    q, n = rand((2, 4, 1, 64)), i32(20, 20)
    need = fa.decode_workspace_bytes(2, 4, 2, 64)
    one = torch.empty(16, dtype=torch.uint8, device="cuda")
    strided = torch.empty(2 * need, dtype=torch.uint8, device="cuda")
    for ws in (one[:1].expand(need), one[None].expand(need // 16 + 1, 16), strided[::2], strided.view(2, need).t()):
        with pytest.raises(ValueError, match="workspace"):
            fa.decode_attention(q, cache, table, n, workspace=ws)
    fa.decode_attention(q, cache, table, n, workspace=strided)
    torch.cuda.synchronize()


def test_attention_calls_refuse_a_workspace_that_is_not_contiguous():
    fa = fa_module()
    q, k, v = (rand((1, 2, 256, 64), seed=s) for s in range(3))
    bm = fa.create_block_mask(fa.FA_MASK_CAUSAL, None, None, 256, 256)
    out, lse = fa.flex_attention(q, k, v, bm)
    bad = torch.empty(16, dtype=torch.uint8, device="cuda")[:1].expand(1 << 24)
    with pytest.raises(ValueError, match="workspace"):
        fa.flex_attention_backward(q, k, v, out, lse, rand(q.shape, seed=3), bm, workspace=bad)
    pools = [rand((64, 2, 128, 64), seed=s) for s in range(2)]
    table = torch.arange(64, dtype=torch.int32, device="cuda")[None]
    one = fa.create_block_mask(fa.FA_MASK_CAUSAL, None, None, 1, 64 * 128)
    with pytest.raises(ValueError, match="workspace"):
        fa.flex_attention(q[:, :, :1].contiguous(), *pools, one, page_table=table, workspace=bad)
    torch.cuda.synchronize()


# ---------------------------------------------------------------- infinities in 16-bit caches

@pytest.mark.parametrize("lens", [NARROW, WIDE], ids=["narrow", "wide"])
@pytest.mark.parametrize("kind, D, group", [("bf16", 128, 1), ("f16", 64, 3), ("f16", 128, 12), ("bf16", 64, 9)])
def test_decode_infinite_values_stay_infinite(kind, D, group, lens):
    # sum p v of a value +inf is +inf however small its weight (here at least e^-30), -inf likewise,
    # NaN where both meet; other elements, heads and sequences are as without them.
    fa = fa_module()
    cache, table, K, V = random_cache(kind, lens, 16, 2, D, seed=group)
    for b, n in enumerate(lens):
        for key in {0, n // 2, n - 1}:
            put(cache, table, b, key, 1, 3, math.inf)
            put(cache, table, b, key, 1, D - 1, -math.inf)
        put(cache, table, b, 0, 1, 8, math.inf)
        put(cache, table, b, n - 1, 1, 8, -math.inf)
        V[b][1][:, [3, 8, D - 1]] = 0
    q = rand((len(lens), 2 * group, 1, D), TYPES[kind], 9, 1.5)
    out, lse = fa.decode_attention(q, cache, table, i32(*lens))
    hit = out[:, group:, 0]
    assert (hit[..., 3] == math.inf).all() and (hit[..., D - 1] == -math.inf).all()
    assert torch.isnan(hit[1:, :, 8]).all() and (hit[0, :, 8] == -math.inf).all()
    hit[..., [3, 8, D - 1]] = 0
    check_decode(q, out, lse, K, V, lens, kind=kind)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_decode_infinite_values_with_light_weights(kind):
    # Weights from 1 down to 2^-60: far below what fp16 holds.
    fa = fa_module()
    for n in (40, 2000):
        cache, table, _, _ = random_cache(kind, [n], 16, 1, 64, seed=n)
        cache.k.zero_()
        cache.v.copy_(torch.zeros_like(cache.v))
        for i in range(n):                       # score of key i: -(i % 61) ln 2
            cache.k[table[0, i // 16].item(), 0, i % 16, 0] = -(i % 61) / 4.0
        q = torch.zeros(1, 1, 1, 64, dtype=TYPES[kind], device="cuda")
        q[..., 0] = 1.0
        for i in range(40):
            put(cache, table, 0, i, 0, i, math.inf if i % 2 else -math.inf)
        out, lse = fa.decode_attention(q, cache, table, i32(n), scale=4 * math.log(2.0))
        want = torch.tensor([math.inf if i % 2 else -math.inf for i in range(40)] + [0.0] * 24, device="cuda")
        assert torch.equal(out[0, 0, 0].float(), want), out
        total = sum(2.0 ** -(i % 61) for i in range(n))
        assert abs(float(lse) - math.log(total)) <= 1e-4


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("n", [60, 2000])
def test_decode_masked_infinite_values_and_scores_count_for_nothing(kind, n):
    fa = fa_module()
    cache, table, K, V = random_cache(kind, [n], 16, 1, 64, seed=2, garbage=False)
    q = rand((1, 4, 1, 64), TYPES[kind], 3)
    at = n - 30
    for key in (0, at - 11, at - 1):
        put(cache, table, 0, key, 0, 5, math.inf)
        cache.k[table[0, key // 16].item(), 0, key % 16, 7] = math.inf
    out, lse = fa.decode_attention(q, cache, table, i32(n), window=30)
    check_decode(q, out, lse, K, V, [n], 30, kind=kind)


# ---------------------------------------------------------------- the largest values

@pytest.mark.parametrize("lens", [[500] * 8, MANY], ids=["narrow", "split"])
def test_decode_largest_bf16_values(lens):
    # A key some e^4 above the others whose values are bf16's largest: its weight times the value is
    # within fp32 as long as no weight exceeds 1.
    fa = fa_module()
    cache, table, _, _ = random_cache("bf16", lens, 16, 2, 64, seed=3, garbage=False)
    cache.k.zero_()
    top = torch.finfo(torch.bfloat16).max
    for b, n in enumerate(lens):
        for h in range(2):
            at = (37 + 61 * b + 29 * h) % n
            cache.k[table[b, at // 16].item(), h, at % 16, 0] = 4.0
            for d in range(64):
                put(cache, table, b, at, h, d, top if d % 2 else -top)
    q = torch.zeros(len(lens), 4, 1, 64, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    out, lse = fa.decode_attention(q, cache, table, i32(*lens), scale=1.0)
    check_decode(q, out, lse, *rows64(cache, table, lens), lens, scale=1.0)


# ---------------------------------------------------------------- row scales over the range of fp32

def scaled_cache(kind, lens, seed, k_log2, v_log2):
    """Pages of 16 for one head; key j's rows have scales 2^k_log2[j] / 64 and 2^v_log2[j] / 64."""
    cache, table, _, _ = random_cache(kind, lens, 16, 1, 64, seed=seed, garbage=False)
    vs = []
    for b, n in enumerate(lens):
        at = torch.arange(n, device="cuda")
        pg, rw = table[b].long()[at // 16], at % 16
        for sc, e in ((cache.k_scale, k_log2), (cache.v_scale, v_log2)):
            sc[pg, 0, rw] = torch.exp2(torch.as_tensor(e, dtype=torch.float32, device="cuda").expand(max(lens))[:n] - 6)
        vs.append(np64(cache.v_scale[pg, 0, rw])[None])
    return cache, table, vs


def check_scaled(q, out, lse, cache, table, lens, kind, vs, scale=None):
    K, V = rows64(cache, table, lens)
    for b in range(len(lens)):
        check_decode(q[b:b + 1], out[b:b + 1], lse[b:b + 1], K[b:b + 1], V[b:b + 1], lens[b:b + 1], scale=scale, kind=kind,
                     vscale=vs[b])


SPREAD = pytest.mark.parametrize("lens", [[300, 500], MANY], ids=["narrow", "split"])


@SPREAD
@pytest.mark.parametrize("kind", ["s8", "e4m3"])
@pytest.mark.parametrize("e", [-120, -100, -60, 0, 60, 108, 119, 125])
def test_decode_value_scales_of_any_size(kind, lens, e):
    # One key at the top, the others 2^-15 of it: lse does not depend on the values, and the result
    # scales with them.
    fa = fa_module()
    cache, table, vs = scaled_cache(kind, lens, 7, 0.0, float(e))
    cache.k.view(torch.uint8).zero_()
    for b, n in enumerate(lens):
        at = 17 * b % n
        cache.k[table[b, at // 16].item(), 0, at % 16, 0] = torch.tensor(64.0).to(cache.dtype)
    q = torch.zeros(len(lens), 3, 1, 64, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 10.4375
    out, lse = fa.decode_attention(q, cache, table, i32(*lens), scale=1.0)
    check_scaled(q, out, lse, cache, table, lens, kind, vs, 1.0)
    assert out.float().abs().amax((1, 2, 3)).min() > 0


@SPREAD
@pytest.mark.parametrize("kind", ["s8", "e4m3"])
@pytest.mark.parametrize("lo, hi", [(-120, 110), (90, 125), (-120, -80), (-40, 40)])
def test_decode_value_scales_of_all_sizes_together(kind, lens, lo, hi):
    fa = fa_module()
    e = torch.randint(lo, hi + 1, (max(lens),), generator=torch.Generator().manual_seed(hi)).float()
    cache, table, vs = scaled_cache(kind, lens, 8, 0.0, e)
    q = rand((len(lens), 4, 1, 64), seed=5, scale=2.0)
    out, lse = fa.decode_attention(q, cache, table, i32(*lens))
    check_scaled(q, out, lse, cache, table, lens, kind, vs)


@SPREAD
@pytest.mark.parametrize("kind", ["s8", "e4m3"])
def test_decode_zero_scales_beside_others(kind, lens):
    # Scales of 0, as fresh pools hold them, among ordinary and tiny ones: their rows are zeros.
    fa = fa_module()
    e = torch.zeros(max(lens))
    e[::3], e[1::3], e[:64] = -math.inf, -110.0, -math.inf
    cache, table, vs = scaled_cache(kind, lens, 9, 0.0, e)
    q = rand((len(lens), 4, 1, 64), seed=6, scale=3.0)
    out, lse = fa.decode_attention(q, cache, table, i32(*lens))
    check_scaled(q, out, lse, cache, table, lens, kind, [np.maximum(v, 2.0 ** -116) for v in vs])


@SPREAD
@pytest.mark.parametrize("kind", ["s8", "e4m3"])
@pytest.mark.parametrize("e", [-100, -30, 60, 100, 112])
def test_decode_key_scales_of_any_size(kind, lens, e):
    # Large keys under a small query: the scores are ordinary numbers.
    fa = fa_module()
    cache, table, vs = scaled_cache(kind, lens, 10, float(e), 0.0)
    q = (rand((len(lens), 4, 1, 64), torch.float32, 7) * 2.0 ** -min(e, 100)).to(torch.bfloat16)
    scale = 2.0 ** (min(e, 100) - e) / 8.0
    out, lse = fa.decode_attention(q, cache, table, i32(*lens), scale=scale)
    check_scaled(q, out, lse, cache, table, lens, kind, vs, scale)


@pytest.mark.parametrize("lens", [[300, 60], [3000, 60]], ids=["narrow", "wide"])
@pytest.mark.parametrize("kind", ["s8", "e4m3"])
@pytest.mark.parametrize("late", [False, True])
@pytest.mark.parametrize("zeros", [False, True])
def test_decode_rows_that_held_no_numbers(kind, lens, late, zeros):
    # A value row whose scale is NaN (as one written with a NaN or an infinity has, beside codes 0)
    # makes its head's outputs NaN, but not lse.
    fa = fa_module()
    cache, table, _, _ = random_cache(kind, lens, 16, 2, 64, seed=4, garbage=False)
    q = rand((2, 6, 1, 64), seed=3)
    clean, lse = fa.decode_attention(q, cache, table, i32(*lens))
    at = lens[0] - 2 if late else 0
    page = table[0, at // 16].item()
    cache.v_scale[page, 1, at % 16] = math.nan
    if zeros:
        cache.v.view(torch.uint8)[page, 1, at % 16] = 0
    out, lse2 = fa.decode_attention(q, cache, table, i32(*lens))
    assert torch.isnan(out[0, 3:]).all() and torch.isfinite(out[0, :3]).all()
    assert torch.equal(out[1], clean[1]) and torch.equal(lse2, lse)


@SPREAD
@pytest.mark.parametrize("kind", ["s8", "e4m3"])
def test_decode_scores_of_zero_under_large_factors(kind, lens):
    # Queries and key scales whose product leaves fp32, met by codes of zero: the scores are zero.
    fa = fa_module()
    cache, table, vs = scaled_cache(kind, lens, 11, 100.0, 0.0)
    cache.k.view(torch.uint8)[..., :32] = 0
    q = torch.zeros(len(lens), 3, 1, 64, dtype=torch.bfloat16, device="cuda")
    q[..., :32] = 2.0 ** 120
    out, lse = fa.decode_attention(q, cache, table, i32(*lens))
    q.zero_()
    check_scaled(q, out, lse, cache, table, lens, kind, vs)


# ---------------------------------------------------------------- reads out of range

@pytest.mark.parametrize("kind", ["s8", "bf16"])
def test_read_records_lengths_and_starts_out_of_range(kind):
    # Each the only fault of its call; what is in range is read all the same.
    fa = fa_module()
    cache = make_cache(kind, 4, 2, 16, 64)
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    x = rand((2, 2, 32, 64), seed=1)
    fa.cache_append(cache, x, x, table, i32(0, 0))
    whole, _ = fa.cache_read(cache, table, i32(32, 32), 32)
    assert fa.cache_status() == fa.FA_OK
    bad = fa.FA_ERR_INVALID_ARG
    k, _ = fa.cache_read(cache, table, i32(20, -1), 8)
    assert fa.cache_status() == bad and torch.equal(k[0], whole[0, :, :8]) and not k[1].any()
    k, _ = fa.cache_read(cache, table, i32(33, 20), 8)
    assert fa.cache_status() == bad and torch.equal(k, whole[:, :, :8])
    k, v = fa.cache_read(cache, table, i32(33, 20), 40)
    assert fa.cache_status() == bad and torch.equal(k[0, :, :32], whole[0]) and not v[0, :, 32:].any()
    k, _ = fa.cache_read(cache, table, i32(20, 20), 8, start=i32(0, -2))
    assert fa.cache_status() == bad and torch.equal(k[0], whole[0, :, :8])
    assert not k[1, :, :2].any() and torch.equal(k[1, :, 2:], whole[1, :, :6])
    k, _ = fa.cache_read(cache, table, i32(20, 20), 8, start=i32(0, -100))
    assert fa.cache_status() == bad and not k[1].any()
    k, _ = fa.cache_read(cache, table, i32(0, 32), 8, start=i32(50, 40))         # past the length: zeros, no fault
    assert fa.cache_status() == fa.FA_OK and not k.any()


# ---------------------------------------------------------------- frequencies

@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", [64, 24, 26])
def test_rotary_frequencies_that_are_no_numbers(inter, rot):
    # Their pairs are NaN at every position, as cos and sin of a product with them are; others stay.
    fa = fa_module()
    f = fa.rotary_frequencies(rot)
    f[1], f[4], f[rot // 2 - 1] = math.nan, math.inf, -math.inf
    x = rand((2, 3, 9, 64), seed=1)
    pos = torch.arange(9, device="cuda", dtype=torch.int32)
    y, _ = fa.rotary(x, None, pos, f, interleaved=inter)
    bad = ~torch.isfinite(f)
    at = torch.nonzero(bad).flatten().tolist()
    hit = sorted(2 * i for i in at) + sorted(2 * i + 1 for i in at) if inter else at + [i + rot // 2 for i in at]
    assert torch.isnan(y[..., hit]).all()
    f[bad] = 0.0
    y[..., hit] = x[..., hit]
    check_rotary(x, y, np.tile(np64(pos), (2, 1)), f, inter, 1.0)


# ---------------------------------------------------------------- the status

def test_status_is_shared_by_streams_and_taken_once():
    # Faults of the rows' calls and of decode, on two streams; each is seen by exactly one look, and what
    # is recorded between two looks is the second one's.
    fa = fa_module()
    cache, table, _, _ = random_cache("s8", [20, 20], 16, 2, 64)
    q, n, long = rand((2, 4, 1, 64)), i32(20, 20), i32(20, 5000)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    calls = (lambda: fa.decode_attention(q, cache, table, long), lambda: fa.cache_read(cache, table, long, 4))
    for first in range(2):
        for both in (False, True):
            with torch.cuda.stream(streams[first]):
                calls[first]()
                if both:
                    calls[1 - first]()
            torch.cuda.synchronize()
            assert fa.cache_status(streams[1 - first]) == fa.FA_ERR_INVALID_ARG
            assert fa.cache_status(streams[first]) == fa.FA_OK
            with torch.cuda.stream(streams[first]):
                fa.decode_attention(q, cache, table, n)
            assert fa.cache_status(streams[first]) == fa.FA_OK


def test_status_loses_nothing_under_concurrent_looks():
    # One thread polls one stream while another records a fault on a second stream and waits for it:
    # every fault has to be seen by a look that ends after it.
    import threading
    fa = fa_module()
    cache, table, _, _ = random_cache("s8", [20, 20], 16, 2, 64)
    long = i32(20, 5000)
    side, poll = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    seen, stop = [0], threading.Event()

    def look():
        while not stop.is_set():
            seen[0] += fa.cache_status(poll) != fa.FA_OK

    thread = threading.Thread(target=look)
    thread.start()
    try:
        for _ in range(200):
            before = seen[0]
            with torch.cuda.stream(side):
                fa.cache_read(cache, table, long, 4)
            side.synchronize()
            for _ in range(20000):
                if seen[0] > before:
                    break
                stop.wait(0.0005)
            assert seen[0] > before
    finally:
        stop.set()
        thread.join()
    assert fa.cache_status() == fa.FA_OK


# ---------------------------------------------------------------- bad pages and lengths where keys are split

@pytest.mark.parametrize("kind, D", [("bf16", 64), ("f16", 128), ("s8", 128), ("e4m3", 64)])
@pytest.mark.parametrize("B, H, G", [(4, 2, 4), (12, 4, 10), (36, 8, 8)], ids=["few", "more", "many"])
def test_decode_bad_pages_and_lengths_over_wide_tables(kind, D, B, H, G):
    # Tables of more than 1024 tokens, so the keys of a head are split over warps and their parts are
    # joined (in three ways, by the number of heads).  A bad page's keys count for nothing; a run of
    # bad pages leaves parts, or a whole sequence, without a key; too long a length ends at the table.
    fa = fa_module()
    page = 32
    lens = [1200 + (997 * b) % 1500 for b in range(B)]
    cache, table, K, V = random_cache(kind, lens, page, H, D, seed=B)
    width = -(-max(lens) // page)
    table = table[:, :width].contiguous()
    g = torch.Generator().manual_seed(B)
    keep = [np.ones(n, dtype=bool) for n in lens]

    def lose(b, j, index):
        table[b, j] = index
        keep[b][j * page:(j + 1) * page] = False

    for b, n in enumerate(lens):
        pages = -(-n // page)
        if b % 4 == 1:
            for j in range(pages):                       # all
                lose(b, j, -1 - j)
        elif b % 4 == 2:
            for j in range(pages // 5, pages // 2):      # one run
                lose(b, j, cache.n_pages)
        elif b % 4 == 3:
            for j in torch.randperm(pages, generator=g)[:pages // 3].tolist() + [pages - 1]:
                lose(b, j, 2 ** 30 + j)
    said = list(lens)
    said[0] = width * page + 1                           # longer than the table: all that it maps
    long = width * page
    table[0] = table[0].clamp(0, cache.n_pages - 1)
    for w, into in ((0, K), (1, V)):
        into[0] = gather64(cache, table, 0, long, w)
    dead = np.isnan(K[0]).any((0, 2)) | np.isnan(V[0]).any((0, 2))      # pool rows that hold no numbers
    for j in range(long // page):
        if dead[j * page:(j + 1) * page].any():
            table[0, j] = -7
            dead[j * page:(j + 1) * page] = True
    keep[0] = ~dead
    said.append(-5)                                      # a sequence of negative length
    table = torch.cat((table, table[:1]))
    q = rand((B + 1, H * G, 1, D), TYPES["f16" if kind == "f16" else "bf16"], 5, 1.5)
    out, lse = fa.decode_attention(q, cache, table, i32(*said))
    assert fa.cache_status() == fa.FA_ERR_INVALID_ARG and fa.cache_status() == fa.FA_OK
    rows = [[x[b][:, keep[b]] for b in range(B)] for x in (K, V)]
    check_decode(q[:B], out[:B], lse[:B], *rows, [int(k.sum()) for k in keep], kind=kind)
    assert not out[B].any() and torch.isneginf(lse[B]).all()
    said = [0 if b == 0 or not keep[b].all() else n for b, n in enumerate(lens)] + [0]
    fa.decode_attention(q, cache, table, i32(*said))
    assert fa.cache_status() == fa.FA_OK


# ---------------------------------------------------------------- weights

@pytest.mark.parametrize("lens", [[1, 2, 5, 40, 700], [1, 2, 5, 40, 2500]], ids=["narrow", "wide"])
@pytest.mark.parametrize("kind", ["s8", "e4m3"])
@pytest.mark.parametrize("D, G", [(64, 3), (128, 12)])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
def test_decode_weights_over_8_bit_caches(kind, D, G, lens, dt):
    # Two fp16 numbers a weight: 2^-22 of itself, or 2^-25 of the largest where the second number is
    # below fp16's normal range; then the result's one rounding, half a step of it.
    fa = fa_module()
    cache, table, K, V = random_cache(kind, lens, 16, 2, D, seed=G)
    q = rand((len(lens), 2 * G, 1, D), dt, 9, 1.5)
    out, lse = fa.decode_attention(q, cache, table, i32(*lens))
    for b, n in enumerate(lens):
        at = np.arange(n)
        vs = np64(cache.v_scale[table[b].long().cpu().numpy()[at // 16], :, at % 16]).T
        o, _, weight, reach, fine = ref.decode(np64(q[b, :, 0]), K[b], V[b], n, vscale=vs)
        score = D * 2.0 ** -24 * reach + 2e-6 * (1 + reach)              # a score's error, as everywhere
        tol = torch.finfo(dt).eps / 2 * np.abs(o) + (2.0 ** -22 + 2 * score + 1e-5) * weight + 2.0 ** -25 * fine + 2.0 ** -25
        assert (np.abs(np64(out[b, :, 0]) - o) <= tol).all()
