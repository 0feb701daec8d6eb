"""Sizes of the several-query-token calls that must not end the process (CPU only:
each runs in a child, and nothing is launched)."""
import subprocess
import sys

import pytest

import paged_kv_cache_443_b200 as pk
from conftest import ROOT

CHILD = """
import ctypes, sys
sys.path.insert(0, {root!r})
import paged_kv_cache_443_b200 as pk
L, F = pk.lib(), 1 << 20
rule = ctypes.byref(pk._ScoreRule({cap}, {window}, None, None, None))
head = (F, F, F, F, F, 1 << 20, F, F, {B}, {T}, {maxq}, {Hq}, {Hkv}, 128, 16, 100, 0.1, pk.PA_BF16)
tail = ({P}, {ctx}, None, 0, None)
print(L.pa_decode_multi_scored(*head, rule, *tail), L.pa_decode_multi(*head, *tail),
      pk.pa_launch_count())
"""


def statuses(**kw):
    """Status of pa_decode_multi_scored and of pa_decode_multi."""
    from paged_kv_cache_443_b200 import build
    build.build()
    a = dict(cap=30.0, window=0, B=2, T=8, maxq=4, Hq=32, Hkv=8, P=0, ctx=4096)
    a.update(kw)
    r = subprocess.run([sys.executable, "-c", CHILD.format(root=ROOT, **a)], capture_output=True,
                       text=True, timeout=120)
    assert r.returncode == 0, (r.returncode, r.stderr[-300:])
    scored, plain, launches = map(int, r.stdout.split())
    assert launches == 0
    return scored, plain


@pytest.mark.parametrize("window", [0, 700])
@pytest.mark.parametrize("maxq,ctx,Hq", [(512, 4096, 32), (4, 4096, 32), (512, 400, 32), (17, 513, 8),
                                         (1, 4096, 64), (300, 1 << 24, 32)])
def test_an_empty_batch_is_nothing_to_do(window, maxq, ctx, Hq):
    assert statuses(B=0, T=0, maxq=maxq, ctx=ctx, Hq=Hq, window=window) == (pk.PA_OK, pk.PA_OK)
    assert statuses(B=3, T=0, maxq=maxq, ctx=ctx, Hq=Hq, window=window) == (pk.PA_OK, pk.PA_OK)


@pytest.mark.parametrize("Hq,Hkv", [(256, 1), (1024, 2), (2000, 2), (1 << 20, 8)])
@pytest.mark.parametrize("B,T,maxq,ctx", [(2, 8, 4, 4096), (0, 0, 512, 4096), (4, 600, 512, 1 << 20)])
def test_heads_per_kv_head_past_a_query_block_are_refused(Hq, Hkv, B, T, maxq, ctx):
    want = (pk.PA_ERR_UNSUPPORTED, pk.PA_ERR_UNSUPPORTED)
    assert statuses(Hq=Hq, Hkv=Hkv, B=B, T=T, maxq=maxq, ctx=ctx) == want
    assert statuses(Hq=Hq, Hkv=Hkv, B=B, T=T, maxq=maxq, ctx=ctx, window=700) == want


@pytest.mark.parametrize("maxq", [2 ** 31 - 1, 2 ** 31 - 127, 0, -5, -2 ** 31])
@pytest.mark.parametrize("window", [0, 700])
def test_query_lengths_out_of_range(maxq, window):
    assert statuses(maxq=maxq, window=window) == (pk.PA_ERR_INVALID, pk.PA_ERR_INVALID)
    assert statuses(maxq=maxq, window=window, T=0) == (pk.PA_OK, pk.PA_OK)
