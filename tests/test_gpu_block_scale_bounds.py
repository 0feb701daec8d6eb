"""Stored scales outside [2^-40, 2^80] (a caller's own): the append takes them as the
decode reads them, so that what it writes beside them and what it keeps of older
codes come back as they were given."""
import numpy as np
import pytest
import torch

import paged_kv_cache_443_b200 as pk
from operators_ref import e4m3_decode, e4m3_encode

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn
LOW, HIGH = 2.0 ** -40, 2.0 ** 80


@pytest.fixture(autouse=True)
def clean_status():
    pk.pa_device_status(clear=True)
    yield
    torch.cuda.synchronize()
    assert pk.pa_device_status() == 0


STORED = [2.0 ** 81, 3e24, 1e30, 3e38, float("inf"), 2.0 ** 80, 2.0 ** -41, 2.0 ** -60, 1e-45, 1e-38,
          2.0 ** -40]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("together", [False, True])
@pytest.mark.parametrize("exponent", [-36, -33, 0, 85])
def test_stored_scales_out_of_bounds(dtype, dim, together, exponent):
    """together: the blocks' tokens in one call and one warp, else a call each.  The new
    elements reach from 2^exponent to about 2^(exponent + 4)."""
    gen = torch.Generator().manual_seed(exponent + 50)
    n, bs = len(STORED), 16
    codes = e4m3_encode((torch.randn(n, 1, bs, dim, generator=gen) * 90).numpy())
    stored = np.array(STORED, dtype=np.float32).reshape(n, 1)
    k, v = (torch.from_numpy(codes.copy()).cuda() for _ in range(2))
    ks, vs = (torch.from_numpy(stored.copy()).cuda() for _ in range(2))
    x = (torch.exp2(4 * torch.rand(n, 1, dim, generator=gen) + exponent) *
         torch.where(torch.rand(n, 1, dim, generator=gen) < 0.5, -1.0, 1.0)).to(dtype)
    slots = torch.tensor([b * bs + 3 + b % 5 for b in range(n)])
    calls = [slice(0, n)] if together else [slice(b, b + 1) for b in range(n)]
    for c in calls:
        pk.pa_reshape_and_cache_fp8_block(x[c].cuda(), x[c].cuda(), k.view(F8), v.view(F8), ks, vs,
                                          slots[c].cuda())
    for got, scales in ((k, ks), (v, vs)):
        got, scales = got.cpu().numpy(), scales.cpu().double().numpy()[:, 0]
        for b in range(n):
            old = min(max(STORED[b], LOW), HIGH)              # as pa_decode_fp8_block reads them
            now = min(max(scales[b], LOW), HIGH)
            most = float(x[b].abs().max())
            need = min(max(2.0 ** np.ceil(np.log2(most / 448)), LOW), HIGH)
            assert now == max(old, need)
            at = int(slots[b]) % bs
            others = [o for o in range(bs) if o != at]
            np.testing.assert_array_equal(got[b, 0, at], e4m3_encode(x[b, 0].double().numpy() / now))
            want = e4m3_encode(e4m3_decode(codes[b, 0, others]) * (old / now))
            np.testing.assert_array_equal(got[b, 0, others], want)
