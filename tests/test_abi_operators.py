"""Refusals of the block-scaled cache and score-rule calls, on the host before any
launch (CPU only: no device call is made), and the references' own pins."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_443_b200 as pk
from operators_ref import E4M3, attention, block_scale, e4m3_decode, e4m3_encode, limits

FAKE = 1 << 20
INVALID, UNSUPPORTED = pk.PA_ERR_INVALID, pk.PA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    from paged_kv_cache_443_b200 import build
    build.build()
    return pk.lib()


@pytest.fixture(autouse=True)
def no_launches(L):
    before = pk.pa_launch_count()
    yield
    assert pk.pa_launch_count() == before


def rule(softcap=0.0, window=0, slopes=None, starts=None, prefix=None):
    return ctypes.byref(pk._ScoreRule(softcap, window, slopes, starts, prefix))


COMMON_BAD = [
    (dict(dtype=7), INVALID), (dict(dtype=pk.PA_FP8_E4M3), UNSUPPORTED), (dict(B=-1), INVALID),
    (dict(Hq=6, Hkv=4), INVALID), (dict(Hq=32, Hkv=2), UNSUPPORTED), (dict(D=96), UNSUPPORTED),
    (dict(D=0), INVALID), (dict(bs=64), UNSUPPORTED), (dict(bs=0), INVALID), (dict(NB=0), INVALID),
    (dict(maxb=0), INVALID), (dict(P=100), INVALID), (dict(maxctx=-1), INVALID),
    (dict(maxctx=8 * 16 + 1), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(q=None), INVALID), (dict(out=FAKE + 8), INVALID), (dict(tables=FAKE + 2), INVALID),
    (dict(P=32), INVALID), (dict(P=32, ws=FAKE, wsb=64), INVALID),
]


def args(**kw):
    a = dict(out=FAKE, q=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, tables=FAKE, maxb=8, lens=FAKE,
             B=2, Hq=8, Hkv=2, D=128, bs=16, NB=100, scale=0.1, dtype=pk.PA_BF16, P=0, maxctx=100,
             ws=None, wsb=0, rule=rule(softcap=30.0), qs=FAKE, T=6, maxq=4)
    a.update(kw)
    return a


def decode_block(L, **kw):
    a = args(**kw)
    return L.pa_decode_fp8_block(a["out"], a["q"], a["k"], a["v"], a["ks"], a["vs"], a["tables"],
                                 a["maxb"], a["lens"], a["B"], a["Hq"], a["Hkv"], a["D"], a["bs"],
                                 a["NB"], a["scale"], a["dtype"], a["P"], a["maxctx"], a["ws"],
                                 a["wsb"], None)


def scored(L, **kw):
    a = args(**kw)
    return L.pa_decode_scored(a["out"], a["q"], a["k"], a["v"], a["tables"], a["maxb"], a["lens"],
                              a["B"], a["Hq"], a["Hkv"], a["D"], a["bs"], a["NB"], a["scale"],
                              a["dtype"], a["rule"], a["P"], a["maxctx"], a["ws"], a["wsb"], None)


def multi(L, **kw):
    a = args(**kw)
    return L.pa_decode_multi_scored(a["out"], a["q"], a["k"], a["v"], a["tables"], a["maxb"],
                                    a["lens"], a["qs"], a["B"], a["T"], a["maxq"], a["Hq"],
                                    a["Hkv"], a["D"], a["bs"], a["NB"], a["scale"], a["dtype"],
                                    a["rule"], a["P"], a["maxctx"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,want", COMMON_BAD + [
    (dict(ks=None), INVALID), (dict(vs=None), INVALID), (dict(ks=FAKE + 2), INVALID)])
def test_decode_fp8_block_refuses(L, kw, want):
    assert decode_block(L, **kw) == want and pk.pa_last_error()


BAD_RULES = [
    dict(rule=rule(softcap=-1.0)), dict(rule=rule(softcap=float("inf"))),
    dict(rule=rule(softcap=float("nan"))), dict(rule=rule(softcap=1e-44)),
    dict(rule=rule(window=-1)), dict(rule=rule(slopes=FAKE + 2)),
    dict(rule=rule(starts=FAKE + 1)), dict(rule=rule(prefix=FAKE + 3)),
]


@pytest.mark.parametrize("cap", [1048577.0, 3e38])
def test_caps_past_the_precision_of_a_score_are_refused(L, cap):
    assert scored(L, rule=rule(softcap=cap)) == INVALID
    assert multi(L, rule=rule(softcap=cap)) == INVALID


def test_rule_values_past_a_c_type():
    """A window of more than 2^31 positions is all of them, not what a C int leaves of it;
    a softcap below the least float32 is not "no cap"."""
    q = torch.zeros(1, 2, 128)
    for window, want in ((2 ** 32 + 5, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1), (-2 ** 32, -1), (7, 7)):
        assert pk.ScoreRule(window=window)._struct(q, 1).window == want
    with pytest.raises(pk.PagedKVError):
        pk.ScoreRule(softcap=1e-60)


def test_pairs_that_the_gpu_cannot_read_are_refused():
    with pytest.raises(pk.PagedKVError):
        pk._pairs(torch.zeros(1, 2, dtype=torch.int64))
    assert pk._pairs(torch.zeros(0, 2, dtype=torch.int64)) == (None, 0)


@pytest.mark.parametrize("kw,want", COMMON_BAD + [(r, INVALID) for r in BAD_RULES])
def test_decode_scored_refuses(L, kw, want):
    assert scored(L, **kw) == want and pk.pa_last_error()


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=pk.PA_F32), UNSUPPORTED), (dict(D=64), UNSUPPORTED), (dict(Hq=24), UNSUPPORTED),
    (dict(Hq=15), INVALID), (dict(bs=64), UNSUPPORTED), (dict(P=192), INVALID),
    (dict(maxq=0), INVALID), (dict(maxq=7), INVALID), (dict(maxctx=8 * 16 + 1), INVALID),
    (dict(qs=None), INVALID), (dict(qs=FAKE + 2), INVALID), (dict(q=FAKE + 8), INVALID),
    (dict(maxb=64, maxctx=1000, P=256), INVALID), (dict(scale=float("inf")), INVALID),
] + [(r, INVALID) for r in BAD_RULES])
def test_decode_multi_scored_refuses(L, kw, want):
    assert multi(L, **kw) == want and pk.pa_last_error()


def test_nothing_to_do_is_ok(L):
    assert decode_block(L, B=0) == pk.PA_OK
    assert scored(L, B=0) == pk.PA_OK and scored(L, B=0, rule=None) == pk.PA_OK
    assert multi(L, B=0) == pk.PA_OK and multi(L, T=0) == pk.PA_OK
    assert multi(L, T=0, rule=None) == pk.PA_OK


def test_a_window_needs_the_windows_workspace(L):
    # 8000 tokens in partitions of 512 need split-K partials, a window of 100 does not
    kw = dict(maxb=500, maxctx=8000, P=512)
    assert scored(L, **kw) == INVALID and "workspace" in pk.pa_last_error()
    assert scored(L, **kw, rule=rule(window=512)) == INVALID
    assert scored(L, **kw, rule=rule(window=100), B=0) == pk.PA_OK
    # a prefix seen from everywhere undoes the window's bound for several query tokens
    assert multi(L, **kw, rule=rule(window=100, prefix=FAKE)) == INVALID
    assert "workspace" in pk.pa_last_error()


def test_append_and_copies_refuse(L):
    def app(**kw):
        a = dict(key=FAKE, k=FAKE, ks=FAKE, vs=FAKE, slots=FAKE, N=4, H=2, D=128, bs=16, NB=10,
                 dtype=pk.PA_F16)
        a.update(kw)
        return L.pa_reshape_and_cache_fp8_block(a["key"], FAKE, a["k"], FAKE, a["ks"], a["vs"],
                                                a["slots"], a["N"], a["H"], a["D"], a["bs"],
                                                a["NB"], a["dtype"], None)
    for kw, want in [(dict(dtype=9), INVALID), (dict(dtype=pk.PA_FP8_E4M3), INVALID),
                     (dict(N=-1), INVALID), (dict(D=80), UNSUPPORTED), (dict(bs=12), UNSUPPORTED),
                     (dict(H=0), INVALID), (dict(NB=0), INVALID), (dict(key=None), INVALID),
                     (dict(key=FAKE + 4), INVALID), (dict(k=FAKE + 1), INVALID),
                     (dict(slots=FAKE + 4), INVALID), (dict(ks=None), INVALID),
                     (dict(vs=FAKE + 2), INVALID), (dict(N=1 << 30, H=4), UNSUPPORTED)]:
        assert app(**kw) == want, kw
        assert pk.pa_last_error()
    assert app(N=0) == pk.PA_OK

    def swap(**kw):
        a = dict(dk=FAKE, sk=FAKE, dks=FAKE, sks=FAKE, pairs=FAKE, P=3, D=128, bs=16, dn=5, sn=7)
        a.update(kw)
        return L.pa_swap_blocks_fp8_block(a["dk"], FAKE, a["dks"], FAKE, a["dn"], a["sk"], FAKE,
                                          a["sks"], FAKE, a["sn"], a["pairs"], a["P"], 2, a["D"],
                                          a["bs"], None)
    for kw, want in [(dict(P=-1), INVALID), (dict(dk=None), INVALID), (dict(sks=None), INVALID),
                     (dict(dks=FAKE + 1), INVALID), (dict(pairs=FAKE + 4), INVALID),
                     (dict(sk=FAKE + 8), INVALID), (dict(D=32), UNSUPPORTED),
                     (dict(bs=4), UNSUPPORTED), (dict(dn=0), INVALID), (dict(sn=0), INVALID)]:
        assert swap(**kw) == want, kw
    assert swap(P=0) == pk.PA_OK
    assert L.pa_copy_blocks_fp8_block(FAKE, FAKE, None, FAKE, FAKE, 3, 2, 128, 16, 10, None) == INVALID
    assert L.pa_copy_blocks_fp8_block(FAKE, FAKE, FAKE, FAKE, None, 0, 2, 128, 16, 10, None) == pk.PA_OK


def test_the_binding_refuses(L):
    """Shapes, types and devices, before the library is called."""
    f8 = torch.float8_e4m3fn
    cache = torch.zeros(4, 2, 16, 128, dtype=f8)
    scales = torch.ones(4, 2)
    x = torch.zeros(3, 2, 128, dtype=torch.float16)
    slots = torch.zeros(3, dtype=torch.int64)
    q = torch.zeros(1, 2, 128, dtype=torch.float16)
    lens = torch.ones(1, dtype=torch.int32)
    table = torch.zeros(1, 2, dtype=torch.int32)
    app = lambda **kw: pk.pa_reshape_and_cache_fp8_block(
        kw.get("x", x), x, kw.get("cache", cache), cache, kw.get("scales", scales), scales,
        kw.get("slots", slots))
    for kw in (dict(scales=scales.double()), dict(scales=torch.ones(4, 3)),
               dict(scales=torch.ones(2, 4).t()), dict(slots=slots.int()), dict(slots=slots[:2]),
               dict(x=x.float()), dict(x=x[:, :1]), dict(cache=cache.half()), dict()):
        with pytest.raises(pk.PagedKVError):   # the last: not on the GPU
            app(**kw)
    with pytest.raises(pk.PagedKVError):
        pk.pa_decode_fp8_block(q, q, cache, cache, scales, scales, table, lens, 0.1, 16)
    with pytest.raises(pk.PagedKVError):
        pk.pa_copy_blocks_fp8_block(cache, cache, scales, scales, torch.zeros(1, 2, dtype=torch.int64))
    half = cache.half()
    for r in (pk.ScoreRule(30.0), pk.ScoreRule(alibi_slopes=torch.ones(3)),
              pk.ScoreRule(alibi_slopes=torch.ones(2).double()),
              pk.ScoreRule(key_starts=torch.zeros(2, dtype=torch.int32)),
              pk.ScoreRule(prefix_lens=torch.zeros(1, dtype=torch.int64))):
        with pytest.raises(pk.PagedKVError):
            r._struct(q, 1) if r.softcap == 0 else pk.pa_decode_scored(
                q, q, half, half, table, lens, 0.1, 16, r)


# ---- the references' own pins ----


def test_reference_codes():
    all_codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(all_codes.copy()).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(e4m3_decode(all_codes), want)
    x = np.concatenate([np.random.default_rng(1).standard_normal(50000) * 100,
                        (E4M3[1:] + E4M3[:-1]) / 2, -(E4M3[1:] + E4M3[:-1]) / 2, [0.0, -0.0]])
    x = np.clip(x, -448, 448)
    got = e4m3_encode(x)
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    exact = x.astype(np.float32) == x
    np.testing.assert_array_equal(got[exact], want[exact])
    assert e4m3_encode([1e9, -1e9, np.inf, np.nan]).tolist() == [0x7e, 0xfe, 0x7e, 0x7f]


def test_reference_scale():
    assert block_scale(448.0) == 1.0 and block_scale(np.nextafter(448.0, 500)) == 2.0
    assert block_scale(0.0) == 2.0 ** -40 and block_scale(1e38) == 2.0 ** 80


def test_reference_attention_is_the_softmax():
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(n, h, 64, generator=g, dtype=torch.float64)
               for n, h in ((3, 4), (20, 2), (20, 2)))
    pos = [17, 18, 19]
    out, tol = attention(q, k, v, 0.125, torch.float32, 0.0, pos=pos, last=pos)
    want = torch.nn.functional.scaled_dot_product_attention(
        q.transpose(0, 1)[None], k.repeat_interleave(2, 1).transpose(0, 1)[None],
        v.repeat_interleave(2, 1).transpose(0, 1)[None], scale=0.125,
        attn_mask=torch.arange(20)[None, :] <= torch.tensor(pos)[:, None])[0].transpose(0, 1)
    assert (out - want).abs().max() < 1e-12
    assert float(tol.max()) < 1e-4
    # nothing seen: zeros; a bias that forgets all but the nearest key: its value
    out, _ = attention(q, k, v, 0.125, torch.float32, 0.0, first=[18, 18, 25], last=[17, 18, 19])
    assert bool((out[0] == 0).all()) and bool((out[2] == 0).all())
    assert torch.equal(out[1], v[18].repeat_interleave(2, 0))
    out, _ = attention(q, k, v, 0.125, torch.float32, 0.0, pos=pos, slopes=torch.full((4,), 1e4))
    assert (out - v[17:20].repeat_interleave(2, 1)).abs().max() < 1e-12
    # a cap of almost nothing: the mean
    out, _ = attention(q, k, v, 0.125, torch.float32, 0.0, cap=1e-9)
    assert (out - v.mean(0).repeat_interleave(2, 0)).abs().max() < 1e-8


def test_limits():
    assert limits(10, 9) == (0, 9)
    assert limits(10, 7, window=3) == (5, 7)
    assert limits(10, 7, window=100, key_start=2) == (2, 7)
    assert limits(10, 3, prefix=6) == (0, 5) and limits(10, 3, prefix=60) == (0, 9)
