"""The serving operators without a GPU: refusals of the C entry points before any CUDA call, the
frequency helper, and pins of the float64 oracle."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import serving as ref

from test_abi import _t, fa  # noqa: F401  (the built library as a fixture)


def _cache(fa, k=0x10000, v=0x20000, ks=0x30000, vs=0x40000, dtype=3, page=64, n=8, H=2, D=64, stride=None, sstride=None):
    st = stride or (H * page * D, page * D, D)
    ss = sstride or (H * page, page, 1)
    return fa.FaKvCache(k, v, ks, vs, dtype, page, n, H, D, (ctypes.c_int64 * 3)(*st), (ctypes.c_int64 * 3)(*ss))


def _ref(x):
    return ctypes.byref(x) if x is not None else None


def _append(fa, k, v, c, table=0x1000, ts=4, tw=4, start=0x2000, count=None):
    return fa._lib.fa_cache_append(_ref(k), _ref(v), _ref(c), table, ts, tw, start, count, None)


def _decode(fa, q, c, out, table=0x1000, ts=4, tw=4, lens=0x2000, window=0, kind=0, params=None):
    return fa._lib.fa_decode(_ref(q), _ref(c), table, ts, tw, lens, window, kind, _ref(params), -1.0, _ref(out), None,
                             0x50000, 1 << 30, None)


BAD_CACHES = [
    (dict(dtype=4), "INVALID"), (dict(k=0), "INVALID"), (dict(k=0x10008), "INVALID"), (dict(ks=0), "INVALID"),
    (dict(page=8), "UNSUPPORTED"), (dict(page=48), "UNSUPPORTED"), (dict(page=2048), "UNSUPPORTED"),
    (dict(n=0), "INVALID"), (dict(n=1 << 31), "INVALID"), (dict(H=0), "INVALID"), (dict(D=96), "UNSUPPORTED"),
    (dict(stride=(8192, 4096, 72)), "INVALID"), (dict(stride=(8192, 0, 64)), "INVALID"),
    (dict(sstride=(128, 64, 0)), "INVALID"),
]


@pytest.mark.parametrize("bad, status", BAD_CACHES)
def test_cache_descriptions_are_checked(fa, bad, status):
    c = _cache(fa, **bad)
    want = getattr(fa, "FA_ERR_INVALID_ARG" if status == "INVALID" else "FA_ERR_UNSUPPORTED")
    rows = _t(fa, B=1, H=2, S=3, D=64)
    assert _append(fa, rows, rows, c) == want
    assert fa._lib.fa_cache_read(_ref(c), 0x1000, 4, 4, None, 0x2000, _ref(rows), _ref(rows), None) == want
    q = _t(fa, B=1, H=4, S=1, D=64)
    assert _decode(fa, q, c, q) == want


def test_cache_calls_refuse_bad_arguments(fa):
    c, k = _cache(fa), _t(fa, B=1, H=2, S=3, D=64)
    bad = fa.FA_ERR_INVALID_ARG
    assert _append(fa, None, k, c) == bad and _append(fa, k, k, None) == bad
    assert _append(fa, k, _t(fa, B=1, H=2, S=4, D=64), c) == bad              # lengths differ
    assert _append(fa, _t(fa, B=1, H=3, S=3, D=64), _t(fa, B=1, H=3, S=3, D=64), c) == bad
    assert _append(fa, k, k, c, table=None) == bad
    assert _append(fa, k, k, c, ts=3, tw=4) == bad
    assert _append(fa, k, k, c, start=None) == bad
    assert _append(fa, k, k, _cache(fa, dtype=0)) == bad                      # bf16 rows, fp16 cache
    assert "own dtype" in fa.fa_last_error_message()
    none = _t(fa, B=0, H=2, S=3, D=64, data=0)
    assert _append(fa, none, none, c, table=None, start=None) == fa.FA_OK     # nothing to write


def test_decode_refuses_bad_arguments(fa):
    c, q = _cache(fa), _t(fa, B=1, H=4, S=1, D=64)
    bad = fa.FA_ERR_INVALID_ARG
    assert _decode(fa, _t(fa, B=1, H=4, S=2, D=64), c, _t(fa, B=1, H=4, S=2, D=64)) == bad
    assert _decode(fa, _t(fa, B=1, H=3, S=1, D=64), c, _t(fa, B=1, H=3, S=1, D=64)) == bad    # 3 heads over 2
    assert _decode(fa, _t(fa, B=1, H=4, S=1, D=128), c, _t(fa, B=1, H=4, S=1, D=128)) == bad
    assert _decode(fa, q, c, _t(fa, B=1, H=4, S=1, D=64, dtype=0)) == bad
    assert _decode(fa, q, c, q, window=-1) == bad
    assert _decode(fa, q, c, q, kind=4) == bad and _decode(fa, q, c, q, kind=1) == bad
    assert _decode(fa, q, c, q, kind=1, params=fa.FaScoreParams(0.0, None)) == bad
    assert _decode(fa, q, c, q, lens=None) == bad
    assert _decode(fa, q, _cache(fa, dtype=0), q) == bad
    big = _t(fa, B=65536, H=4, S=1, D=64)
    assert _decode(fa, big, c, big) == fa.FA_ERR_UNSUPPORTED
    many = _t(fa, B=1, H=1025, S=1, D=64)
    assert _decode(fa, many, _cache(fa, H=1), many) == fa.FA_ERR_UNSUPPORTED
    assert fa.decode_workspace_bytes(1, 1025, 1, 64) == 0
    assert fa.decode_workspace_bytes(0, 4, 2, 64) == 0 and fa.decode_workspace_bytes(1, 3, 2, 64) == 0


def test_rotary_refuses_bad_arguments(fa):
    def call(q, k=None, qo=None, ko=None, pos=None, ps=0, f=0x1000, rot=64, layout=0):
        return fa._lib.fa_rotary(_ref(q), _ref(k), pos, ps, 0, f, rot, layout, 1.0, 0, _ref(qo), _ref(ko), None)
    q, bad = _t(fa), fa.FA_ERR_INVALID_ARG
    assert call(None, qo=q) == bad and call(q) == bad
    assert call(q, k=q, qo=q) == bad                                          # k without k_out
    assert call(q, qo=_t(fa, S=128)) == bad
    assert call(q, k=_t(fa, S=128), qo=q, ko=_t(fa, S=128)) == bad
    assert call(q, qo=q, rot=3) == bad and call(q, qo=q, rot=0) == bad and call(q, qo=q, rot=66) == bad
    assert call(q, qo=q, layout=2) == bad and call(q, qo=q, ps=-1) == bad
    assert call(q, qo=_t(fa, stride=(64 * 512, 64, 128, 1))) == bad           # in place, other strides
    assert call(q, qo=q, f=None) == bad
    wide = _t(fa, D=1032)
    assert call(wide, qo=wide) == fa.FA_ERR_UNSUPPORTED
    none = _t(fa, B=0, data=0)
    assert call(none, qo=none, f=None) == fa.FA_OK


def test_binding_refuses_what_the_library_cannot_see(fa):
    k = torch.zeros(2, 1, 16, 64, dtype=torch.int8)
    with pytest.raises(ValueError):
        fa.PagedKVCache(k, k)                                                 # not CUDA, no scales
    with pytest.raises(TypeError):
        fa.PagedKVCache(k.float(), k.float())
    q = torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.rotary(q, None, 0, torch.zeros(32, dtype=torch.float64))


@pytest.mark.parametrize("kind", ["none", "linear", "base", "by_parts"])
@pytest.mark.parametrize("rot", [4, 24, 64, 128])
def test_frequencies(fa, kind, rot):
    code = {"none": fa.FA_ROTARY_SCALE_NONE, "linear": fa.FA_ROTARY_SCALE_LINEAR, "base": fa.FA_ROTARY_SCALE_BASE,
            "by_parts": fa.FA_ROTARY_SCALE_BY_PARTS}[kind]
    got = fa.rotary_frequencies(rot, 10000.0, scaling=code, factor=8.0, original_len=4096, device="cpu").numpy()
    want = ref.rotary_frequencies(rot, 10000.0, kind, 8.0, 4096.0)
    # pow of two libraries, a few units in the last place of float64 each, times rot in base's power
    np.testing.assert_allclose(got, want, rtol=1e-13)
    if kind == "by_parts":
        plain = ref.rotary_frequencies(rot)
        assert got[0] == plain[0] and (rot < 64 or got[-1] == plain[-1] / 8.0)


def test_frequencies_refuse_bad_arguments(fa):
    for bad in (dict(rot_dim=3), dict(rot_dim=0), dict(base=0.0), dict(base=math.inf), dict(scaling=9),
                dict(scaling=fa.FA_ROTARY_SCALE_LINEAR, factor=0.0),
                dict(scaling=fa.FA_ROTARY_SCALE_BY_PARTS, factor=2.0),
                dict(scaling=fa.FA_ROTARY_SCALE_BY_PARTS, factor=2.0, original_len=10, low_turns=4, high_turns=4),
                dict(rot_dim=2, scaling=fa.FA_ROTARY_SCALE_BASE, factor=2.0)):
        with pytest.raises(fa.FaError):
            fa.rotary_frequencies(**{"rot_dim": 64, "device": "cpu", **bad})


def test_oracle_rotary_turns_pairs_and_its_inverse_undoes_them():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((2, 3, 5, 24))
    f = ref.rotary_frequencies(16)
    pos = rng.integers(-50, 10 ** 6, (2, 5))
    for inter in (False, True):
        y = ref.rotary(x, pos, f, inter, 1.5)
        assert np.array_equal(y[..., 16:], x[..., 16:])
        i, j = (2, 3) if inter else (1, 9)                                    # pair 1
        z = (x[..., i] + 1j * x[..., j]) * 1.5 * np.exp(1j * pos[:, None] * f[1])
        np.testing.assert_allclose(y[..., i], z.real, atol=1e-12)
        np.testing.assert_allclose(y[..., j], z.imag, atol=1e-12)
        np.testing.assert_allclose(ref.rotary(y, pos, f, inter, 1 / 1.5, inverse=True), x, atol=1e-12)


def test_oracle_e4m3_rounding_is_the_types():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    codes = np.unique(codes[torch.isfinite(codes)].double().numpy())
    rng = np.random.default_rng(1)
    y = np.concatenate([rng.uniform(-448, 448, 4000), rng.uniform(-0.05, 0.05, 4000), codes, (codes[1:] + codes[:-1]) / 2])
    got = ref.round_e4m3(y)
    assert np.isin(got, codes).all()
    assert (np.abs(got - y) <= np.abs(codes[None] - y[:, None]).min(1)).all()
    assert np.array_equal(got, torch.from_numpy(y).to(torch.float32).to(torch.float8_e4m3fn).double().numpy())


def test_oracle_scales():
    v, s = ref.quantise_s8(np.array([[127.0, -63.5, 64.5, 1.0], [0, 0, 0, 0], [1, np.nan, 0, 0]]))
    assert np.array_equal(v[0], [127, -64, 64, 1]) and s[0] == 1.0 and s[1] == 2.0 ** -126 and np.isnan(s[2])
    v, s = ref.quantise_e4m3(np.array([[448.0, 1.0], [449.0, 1.0], [224.5, 1], [2.0 ** -120, 0]]))
    assert list(s) == [1.0, 2.0, 1.0, 2.0 ** -126]


def test_oracle_decode_is_a_softmax():
    rng = np.random.default_rng(2)
    q, K, V = rng.standard_normal((4, 8)), rng.standard_normal((2, 9, 8)), rng.standard_normal((2, 9, 8))
    out, lse, weight, reach, fine = ref.decode(q, K, V, 7, window=3)
    x = K[1, 4:7] @ q[3] / math.sqrt(8)
    np.testing.assert_allclose(lse[3], np.log(np.exp(x).sum()))
    np.testing.assert_allclose(out[3], np.exp(x - lse[3]) @ V[1, 4:7])
    p = np.exp(x - lse[3])
    np.testing.assert_allclose(weight[3], p @ np.abs(V[1, 4:7]))
    np.testing.assert_allclose(fine[3], p.max() * np.abs(V[1, 4:7]).sum(0))
    assert reach >= np.abs(x).max()
    out, lse, _, _, _ = ref.decode(q, K, V, 0)
    assert not out.any() and np.isneginf(lse).all()
