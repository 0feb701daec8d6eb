"""PagedKVCache launching on a stream that is not the current one: behind work
that keeps that stream busy, while the current stream allocates and fills tensors
of the sizes that the calls need for themselves."""
import numpy as np
import pytest
import torch

import paged_kv_cache_443_b200 as pk
from operators_ref import U, append, attention, gather, worst
from paged_kv_cache_443_b200.cache import PagedKVCache

pytestmark = pytest.mark.gpu
HEADS, GROUP, DIM, BS = 2, 4, 128, 16
SCALE = DIM ** -0.5


@pytest.fixture(autouse=True)
def clean_status():
    pk.pa_device_status(clear=True)
    yield
    torch.cuda.synchronize()
    assert pk.pa_device_status() == 0


class Busy:
    """Calls on a stream that is behind the host by a tenth of a second each."""

    def __init__(self, kind):
        self.side = torch.cuda.Stream()
        handle = self.side.cuda_stream
        self.given = {"stream": self.side, "handle": handle,
                      "wrapper": type("Wrapper", (), {"cuda_stream": handle})()}[kind]
        self.filled = []

    def __call__(self, call, *nbytes):
        with torch.cuda.stream(self.side):
            torch.cuda._sleep(200_000_000)
        result = call(self.given)
        for n in nbytes:
            self.filled += [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for _ in range(3)]
        return result

    def end(self):
        torch.cuda.current_stream().wait_stream(self.side)
        torch.cuda.synchronize()
        for t in self.filled:
            assert bool((t == 7).all())


def draw(gen, *shape):
    return torch.randn(*shape, generator=gen).to(torch.bfloat16)


@pytest.mark.parametrize("kind", ["stream", "handle", "wrapper"])
def test_attention_on_another_stream(kind):
    gen = torch.Generator().manual_seed(21)
    lens, counts = [1300, 900], [3, 5]
    kv = PagedKVCache(160, BS, HEADS, DIM, torch.bfloat16)
    history = []
    for s, n in enumerate(lens):
        kv.add(s)
        k, v = draw(gen, n, HEADS, DIM), draw(gen, n, HEADS, DIM)
        kv.append([s], [n], k.cuda(), v.cuda())
        history.append((k.double(), v.double()))
    table, length, longest = kv.tables([0, 1])
    q = draw(gen, sum(counts), HEADS * GROUP, DIM)
    one = draw(gen, 2, HEADS * GROUP, DIM)
    start = torch.tensor([0, 3, 8], dtype=torch.int32).cuda()
    dq, done = q.cuda(), one.cuda()
    rule = pk.ScoreRule(softcap=20.0)
    ws_multi = pk.pa_decode_multi_workspace_bytes(8, HEADS * GROUP, DIM, longest)
    ws_one = pk.pa_decode_workspace_bytes(2, HEADS * GROUP, DIM, longest)
    assert ws_multi and ws_one
    torch.cuda.synchronize()
    busy = Busy(kind)
    got = []
    for r in (None, rule):
        got.append(busy(lambda s, r=r: kv.decode_multi(dq, table, length, start, longest, 5, SCALE,
                                                       stream=s, rule=r), ws_multi, q.nbytes))
    for r in (None, rule):
        got.append(busy(lambda s, r=r: kv.decode(done, table, length, longest, SCALE, stream=s,
                                                 rule=r), ws_one, one.nbytes))
    busy.end()
    for i, out in enumerate(got):
        rows = [slice(0, 3), slice(3, 8)] if i < 2 else [slice(0, 1), slice(1, 2)]
        for b, (k, v) in enumerate(history):
            x = (q if i < 2 else one)[rows[b]].double()
            pos = list(range(lens[b] - x.shape[0], lens[b]))
            want, tol = attention(x, k, v, SCALE, torch.bfloat16, U[torch.bfloat16], last=pos,
                                  pos=pos, cap=20.0 if i % 2 else 0.0)
            assert worst(out[rows[b]], want, tol) <= 1, (i, b)


@pytest.mark.parametrize("kind", ["stream", "handle", "wrapper"])
def test_block_scaled_cache_on_another_stream(kind):
    """Append, copy-on-write, swap out and in, decode: uploaded slots and pairs."""
    gen = torch.Generator().manual_seed(22)
    kv = PagedKVCache(200, BS, HEADS, DIM, torch.float8_e4m3fn, block_scales=True)
    kv.enable_swap(100)
    ref = [np.zeros((200, HEADS, BS, DIM), np.uint8) for _ in range(2)] + \
        [np.zeros((200, HEADS), np.float32) for _ in range(2)]
    news = [(draw(gen, n, HEADS, DIM), draw(gen, n, HEADS, DIM) * 2 ** i)
            for i, n in enumerate((1500, 2))]
    dev = [(k.cuda(), v.cuda()) for k, v in news]
    q = draw(gen, 2, HEADS * GROUP, DIM)
    dq = q.cuda()
    kv.add(0)
    torch.cuda.synchronize()
    busy = Busy(kind)

    def store(seqs, counts, i):
        n = sum(counts)
        slots, pairs = busy(lambda s: kv.append(seqs, counts, *dev[i], stream=s), 8 * n, 16)
        for src, dst in pairs:
            for r in ref:
                r[dst] = r[src]
        for x, c, s in zip(news[i], (0, 1), (2, 3)):
            append(x.float().numpy(), ref[c], ref[s], slots)
        return pairs

    store([0], [1500], 0)
    kv.fork(0, 1)
    assert store([0, 1], [1, 1], 1)                  # 1500 = 93 * 16 + 12: a shared block is copied
    out = busy(lambda s: kv.swap_out([1], stream=s), 16 * 94)
    host = {dst: [r[src].copy() for r in ref] for src, dst in out}
    back = busy(lambda s: kv.swap_in([1], stream=s), 16 * 94)
    for src, dst in back:
        for r, h in zip(ref, host[src]):
            r[dst] = h
    table, lens, longest = kv.tables([0, 1])
    ws = pk.pa_decode_workspace_bytes(2, HEADS * GROUP, DIM, longest)
    got = busy(lambda s: kv.decode(dq, table, lens, longest, SCALE, stream=s), ws, q.nbytes)
    busy.end()
    for b in range(2):
        n = int(lens[b])
        row = table[b].cpu()
        have = [gather(c.cpu(), row, n, s.cpu())[0] for c, s in ((kv.k_cache, kv.k_scales),
                                                                (kv.v_cache, kv.v_scales))]
        want = [gather(torch.from_numpy(ref[c]), row, n, torch.from_numpy(ref[c + 2]))
                for c in (0, 1)]
        assert torch.equal(have[0], want[0][0]) and torch.equal(have[1], want[1][0])
        o, tol = attention(q[b:b + 1].double(), have[0], have[1], SCALE, torch.bfloat16, 2.0 ** -8,
                           split=True, floor_values=want[1][1])
        assert worst(got[b], o[0], tol[0]) <= 1
