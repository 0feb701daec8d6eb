"""pa_decode_scored / pa_decode_multi_scored without a rule are the plain calls."""
import pytest
import torch

import paged_kv_cache_443_b200 as pk


class Recorder:
    """Stands for the library: takes every call and keeps the rule it was given."""

    def __init__(self):
        self.rules = []

    def pa_decode_scored(self, *args):
        self.rules.append(args[15])
        return pk.PA_OK

    def pa_decode_multi_scored(self, *args):
        self.rules.append(args[18])
        return pk.PA_OK


def test_the_binding_passes_no_rule_on(monkeypatch):
    lib = Recorder()
    monkeypatch.setattr(pk, "lib", lambda: lib)
    monkeypatch.setattr(pk, "_ready", lambda *tensors: None)
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    cache = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
    table, lens = torch.zeros(2, 2, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    start = torch.tensor([0, 1, 2], dtype=torch.int32)
    pk.pa_decode_scored(q, q, cache, cache, table, lens, 0.1, 16, None, stream=0)
    pk.pa_decode_multi_scored(q, q, cache, cache, table, lens, start, 0.1, 16, 1, None, stream=0)
    assert lib.rules == [None, None]
    pk.pa_decode_scored(q, q, cache, cache, table, lens, 0.1, 16, pk.ScoreRule(30.0), stream=0)
    assert lib.rules[-1] is not None


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,group", [(torch.bfloat16, 8), (torch.float16, 1)])
def test_no_rule_is_the_plain_call(dtype, group):
    gen = torch.Generator().manual_seed(group)
    draw = lambda *shape: torch.randn(*shape, generator=gen).to(dtype).cuda()
    k, v = draw(64, 2, 16, 128), draw(64, 2, 16, 128)
    table = torch.randperm(64, generator=gen)[:50].reshape(2, 25).int().cuda()
    lens = torch.tensor([400, 37], dtype=torch.int32).cuda()
    start = torch.tensor([0, 3, 4], dtype=torch.int32).cuda()
    one, many = draw(2, 2 * group, 128), draw(4, 2 * group, 128)
    out = [torch.empty_like(t) for t in (one, one, many, many)]
    pk.pa_decode(out[0], one, k, v, table, lens, 0.09, 400)
    pk.pa_decode_scored(out[1], one, k, v, table, lens, 0.09, 400, None)
    pk.pa_decode_multi(out[2], many, k, v, table, lens, start, 0.09, 400, 3)
    pk.pa_decode_multi_scored(out[3], many, k, v, table, lens, start, 0.09, 400, 3, None)
    torch.cuda.synchronize()
    assert torch.equal(out[0], out[1]) and torch.equal(out[2], out[3])
    assert pk.pa_device_status() == 0
