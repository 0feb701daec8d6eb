"""Attention under a score rule on the GPU (capped, distance-biased, windowed
scores, documents and prefixes), within the error that the kernels' arithmetic
may leave (operators_ref).  Every position before the first and after the last
that any query of a sequence sees holds NaN or infinities."""
import pytest
import torch

import paged_kv_cache_443_b200 as pk
from operators_ref import attention, gather, limits, worst
from paged_kv_cache_443_b200.cache import PagedKVCache

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_status():
    pk.pa_device_status(clear=True)
    yield
    torch.cuda.synchronize()
    assert pk.pa_device_status() == 0


class Batch:
    """counts: query tokens per sequence (None: the decode call)."""

    def __init__(self, gen, lens, heads, group, bs, dim, dtype, counts=None, rule=None,
                 magnitude=1.0):
        self.lens, self.bs, self.dim, self.dtype = list(lens), bs, dim, dtype
        self.heads, self.group = heads, group
        self.multi = counts is not None
        self.counts = [1] * len(lens) if counts is None else list(counts)
        self.rule = dict(rule or {})
        need = [-(-n // bs) for n in lens]
        blocks = sum(need) + 2
        self.k, self.v = ((torch.randn(blocks, heads, bs, dim, generator=gen) * m).to(dtype)
                          for m in (magnitude, 1.0))
        order = torch.randperm(blocks, generator=gen).int()
        self.table = torch.full((len(lens), max(max(need), 1) + 1), -1, dtype=torch.int32)
        for b, n in enumerate(need):
            self.table[b, :n] = order[sum(need[:b]):sum(need[:b]) + n]
        self.k[order[sum(need):].long()] = float("nan")
        self.v[order[sum(need):].long()] = float("inf")
        rows = sum(self.counts)
        self.q = torch.randn(rows, heads * group, dim, generator=gen).to(dtype)
        # the spans of every query row, and poison outside a sequence's own
        self.spans = []
        row = 0
        for b, n in enumerate(lens):
            spans = []
            for i in range(self.counts[b]):
                pos = n - self.counts[b] + i
                start = self.rule["key_starts"][row] if "key_starts" in self.rule else 0
                prefix = self.rule["prefix_lens"][b] if "prefix_lens" in self.rule else 0
                spans.append((pos, *limits(n, pos, self.rule.get("window", 0), start, prefix)))
                row += 1
            self.spans.append(spans)
            seen = [(first, last) for _, first, last in spans if first <= last]
            low, high = (min(f for f, _ in seen), max(l for _, l in seen)) if seen else (n, -1)
            for j in range(need[b] * bs):
                if not low <= j <= high:
                    blk = int(self.table[b, j // bs])
                    self.k[blk, :, j % bs] = float("nan")
                    self.v[blk, :, j % bs] = float("-inf") if j % 2 else float("nan")

    def score_rule(self):
        as_int = lambda name: torch.tensor(self.rule[name], dtype=torch.int32, device="cuda") \
            if name in self.rule else None
        slopes = self.rule.get("slopes")
        return pk.ScoreRule(self.rule.get("cap", 0.0), self.rule.get("window", 0),
                            slopes.float().cuda() if slopes is not None else None,
                            as_int("key_starts"), as_int("prefix_lens"))

    def run(self, partition=0, scale=None, rule=True, most=None):
        scale = self.dim ** -0.5 if scale is None else scale
        q, k, v, table = (t.cuda() for t in (self.q, self.k, self.v, self.table))
        lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        out = torch.full_like(q, float("nan"))
        longest = max(self.lens)
        size = pk.pa_decode_multi_workspace_bytes if self.multi else pk.pa_decode_workspace_bytes
        n = size(q.shape[0], q.shape[1], self.dim, longest, partition)
        ws = torch.full((n // 4,), float("nan"), device="cuda") if n else None
        kw = dict(partition_size=partition, workspace=ws)
        if not self.multi:
            if rule:
                pk.pa_decode_scored(out, q, k, v, table, lens, scale, longest, self.score_rule(), **kw)
            else:
                pk.pa_decode(out, q, k, v, table, lens, scale, longest, **kw)
            return out
        start = torch.tensor([0] + self.counts, device="cuda").cumsum(0).to(torch.int32)
        args = (out, q, k, v, table, lens, start, scale, longest, most or max(self.counts))
        if rule:
            pk.pa_decode_multi_scored(*args, self.score_rule(), **kw)
        else:
            pk.pa_decode_multi(*args, **kw)
        return out

    def want(self, scale=None):
        scale = self.dim ** -0.5 if scale is None else scale
        tensor_core = self.multi or (self.dtype != torch.float32 and self.dim == 128 and self.group >= 4)
        u_p = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}[self.dtype] if tensor_core else 0.0
        outs, tols, row = [], [], 0
        for b, n in enumerate(self.lens):
            q = self.q[row:row + self.counts[b]].double()
            row += self.counts[b]
            if n == 0 or self.counts[b] == 0:
                outs.append(torch.zeros_like(q))
                tols.append(torch.zeros_like(q))
                continue
            k, v = (gather(t, self.table[b], n) for t in (self.k, self.v))
            pos, first, last = zip(*self.spans[b])
            out, tol = attention(q, k, v, scale, self.dtype, u_p, first=first, last=last, pos=pos,
                                 cap=self.rule.get("cap", 0.0), slopes=self.rule.get("slopes"))
            outs.append(out)
            tols.append(tol)
        return torch.cat(outs), torch.cat(tols)

    def check(self, *partitions, scale=None):
        out, tol = self.want(scale)
        for p in partitions or (0,):
            got = self.run(p, scale).cpu().double()
            assert worst(got, out, tol) <= 1, p


def slopes(n):
    return torch.exp2(-8.0 * torch.arange(1, n + 1) / n)


def rule_for(name, lens, heads):
    return {
        "cap": dict(cap=15.0),
        "slopes": dict(slopes=slopes(heads)),
        "window 1": dict(window=1),
        "window": dict(window=37),
        "window of a partition": dict(window=256, cap=50.0),
        "window past all": dict(window=1 << 30),
        "starts": dict(key_starts=[(i * 53) % (n + 2) - 1 for i, n in enumerate(lens)]),
        "all": dict(cap=30.0, slopes=slopes(heads), window=200,
                    key_starts=[(i * 29) % (n + 9) for i, n in enumerate(lens)]),
    }[name]


RULES = ["cap", "slopes", "window 1", "window", "window of a partition", "window past all",
         "starts", "all"]


@pytest.mark.parametrize("name", RULES)
@pytest.mark.parametrize("dtype,dim,group,heads,bs", [
    (torch.float32, 64, 1, 3, 16), (torch.float32, 128, 8, 1, 8), (torch.float16, 64, 4, 2, 32),
    (torch.float16, 128, 1, 2, 16), (torch.bfloat16, 128, 2, 2, 8),
    (torch.float16, 128, 4, 2, 16), (torch.bfloat16, 128, 8, 1, 32), (torch.bfloat16, 128, 8, 2, 8)])
def test_decode(name, dtype, dim, group, heads, bs):
    gen = torch.Generator().manual_seed(dim + group)
    lens = [0, 1, bs - 1, bs, bs + 1, 36, 37, 38, 127, 128, 129, 255, 256, 257, 513, 900]
    batch = Batch(gen, lens, heads, group, bs, dim, dtype, rule=rule_for(name, lens, heads * group))
    batch.check(0, 128, 256)


@pytest.mark.parametrize("group", [1, 4, 8])
def test_decode_partitions_without_a_multiple_of_a_tile(group):
    gen = torch.Generator().manual_seed(group)
    lens = [700, 33, 1]
    Batch(gen, lens, 2, group, 16, 128, torch.bfloat16,
          rule=rule_for("all", lens, 2 * group)).check(32, 96)


@pytest.mark.parametrize("cap", [1e-3, 2.0, 1e6])
def test_caps_of_any_size(cap):
    """Scores far inside and far past the cap."""
    gen = torch.Generator().manual_seed(1)
    for group in (1, 8):
        Batch(gen, [300, 40], 1, group, 16, 128, torch.float16, rule=dict(cap=cap),
              magnitude=6.0).check()


def test_streamed_partitions():
    """A batch large enough that a CTA takes several partitions, most of them outside
    the window."""
    gen = torch.Generator().manual_seed(3)
    lens = [int(x) for x in torch.randint(1, 1500, (200,), generator=gen)]
    for group, window in ((4, 700), (8, 0), (8, 150)):
        Batch(gen, lens, 2, group, 16, 128, torch.bfloat16,
              rule=dict(cap=20.0, window=window)).check(128)


@pytest.mark.parametrize("dtype,group,heads,bs", [(torch.float16, 4, 2, 16), (torch.bfloat16, 8, 1, 8),
                                                  (torch.bfloat16, 8, 2, 32), (torch.float16, 1, 3, 16),
                                                  (torch.bfloat16, 2, 1, 16)])
@pytest.mark.parametrize("most", [1, 2, 4, 7, 16])
def test_verify(dtype, group, heads, bs, most):
    """A few query tokens per sequence, each with limits of its own."""
    gen = torch.Generator().manual_seed(most + group)
    lens = [most, most + 1, 40, 129, 300, 640, 641]
    counts = [most, 1, max(1, most - 1), most, max(1, most // 2), most, 1]
    rows = sum(counts)
    for rule in (dict(cap=20.0, window=33),
                 dict(slopes=slopes(heads * group), prefix_lens=[0, 30, 100, 5, 1000, -3, 400]),
                 dict(window=5, key_starts=[(i * 17) % 60 for i in range(rows)]),
                 dict(key_starts=[(i * 97) % 700 for i in range(rows)], cap=5.0),
                 dict(key_starts=[1 << 30] * rows)):
        Batch(gen, lens, heads, group, bs, 128, dtype, counts, rule).check(0, 128, 256)


@pytest.mark.parametrize("dtype,group,heads,bs", [(torch.bfloat16, 8, 1, 16), (torch.float16, 4, 2, 8),
                                                  (torch.bfloat16, 2, 2, 32), (torch.float16, 1, 2, 16)])
def test_chunks(dtype, group, heads, bs):
    """Prompt chunks over several query blocks: documents, windows, prefixes."""
    gen = torch.Generator().manual_seed(group)
    lens = [400, 333, 90, 700]
    counts = [400, 77, 1, 290]
    rows = sum(counts)
    docs = []                                 # packed documents of 50, 100, 150 ... tokens
    for n, c in zip(lens, counts):
        starts = [max(s for s in (0, 50, 150, 300, 500) if s <= pos) for pos in range(n - c, n)]
        docs += starts
    for rule in (dict(key_starts=docs), dict(window=64, cap=30.0), dict(window=1),
                 dict(prefix_lens=[150, 400, 0, 600], slopes=slopes(heads * group)),
                 dict(key_starts=[(i * 31) % 800 for i in range(rows)]),
                 dict(prefix_lens=[64, 0, 700, 129], window=100, cap=10.0)):
        Batch(gen, lens, heads, group, bs, 128, dtype, counts, rule).check(0, 128, 384)


def test_extreme_starts_and_prefixes():
    """The extremes of int32: a prefix of none, a document that has not begun."""
    gen = torch.Generator().manual_seed(5)
    least, most = -2 ** 31, 2 ** 31 - 1
    lens = [400, 60, 300]
    for counts in ([4, 1, 3], [200, 60, 3]):
        rows = sum(counts)
        for rule in (dict(prefix_lens=[least, most, least + 1], window=50),
                     dict(prefix_lens=[least, -1, most]),
                     dict(key_starts=[(least, most, 0)[i % 3] for i in range(rows)],
                          prefix_lens=[least, 20, 0], window=most)):
            for group in (1, 8):
                Batch(gen, lens, 1, group, 16, 128, torch.bfloat16, counts, rule).check()
    Batch(gen, lens, 1, 8, 16, 128, torch.bfloat16,
          rule=dict(key_starts=[least, most, most - 1], window=most)).check()


def test_chunk_rows_of_other_sequences_are_left_alone():
    """A sequence without query tokens, and rows past the last sequence's."""
    gen = torch.Generator().manual_seed(9)
    batch = Batch(gen, [300, 200, 100], 1, 8, 16, 128, torch.bfloat16, [70, 0, 100], dict(window=50))
    out, tol = batch.want()
    batch.q = torch.cat([batch.q, torch.zeros(5, 8, 128, dtype=torch.bfloat16)])
    got = batch.run()
    assert worst(got[:170], out, tol) <= 1
    assert bool(got[170:].isnan().all())


@pytest.mark.parametrize("multi", [False, True])
def test_no_rule_is_the_plain_call(multi):
    gen = torch.Generator().manual_seed(2)
    batch = Batch(gen, [700, 33, 1], 2, 4, 16, 128, torch.bfloat16, [3, 2, 1] if multi else None)
    for p in (0, 128):
        assert torch.equal(batch.run(p), batch.run(p, rule=False))


def test_flags_bad_lengths_blocks_and_offsets():
    gen = torch.Generator().manual_seed(4)
    for group in (1, 8):
        batch = Batch(gen, [300, 40], 1, group, 16, 128, torch.float16, rule=dict(window=100))
        out, tol = batch.want()
        batch.table[0, 15] = 10 ** 6          # inside the window
        got = batch.run().cpu().double()
        assert worst(got[1], out[1], tol[1]) <= 1
        assert pk.pa_device_status() == pk.PA_DEVERR_TABLE
        batch.table[0, 15] = -1
        batch.lens[0] = -1
        batch.run()
        assert pk.pa_device_status() == pk.PA_DEVERR_CONTEXT
    for counts in ([5, 2], [200, 2]):
        batch = Batch(gen, [300, 40], 1, 8, 16, 128, torch.float16, counts, dict(window=100))
        out, tol = batch.want()
        batch.lens[1] = 1                     # two query tokens of one
        got = batch.run().cpu().double()
        assert worst(got[:counts[0]], out[:counts[0]], tol[:counts[0]]) <= 1
        assert pk.pa_device_status() == pk.PA_DEVERR_CONTEXT


@pytest.mark.parametrize("counts,rule", [(None, dict(cap=20.0, window=90)), ([4] * 32, dict(window=150)),
                                         ([90] * 32, dict(window=100, cap=10.0))])
def test_repeats_bit_for_bit(counts, rule):
    gen = torch.Generator().manual_seed(6)
    lens = [int(x) for x in torch.randint(100, 700, (32,), generator=gen)]
    batch = Batch(gen, lens, 2, 8, 16, 128, torch.bfloat16, counts, rule)
    one = batch.run(128)
    for _ in range(10):
        assert torch.equal(batch.run(128), one)


def test_cache_serves_a_windowed_model():
    """PagedKVCache: a prompt chunk, then decode steps under one rule, captured into
    a graph and replayed."""
    gen = torch.Generator().manual_seed(12)
    heads, group, dim, bs, n = 2, 4, 128, 16, 150
    cache = PagedKVCache(40, bs, heads, dim, torch.bfloat16)
    cache.add(0)
    kv = [torch.randn(n + 3, heads, dim, generator=gen).to(torch.bfloat16) for _ in range(2)]
    q = torch.randn(n + 3, heads * group, dim, generator=gen).to(torch.bfloat16)
    rule = pk.ScoreRule(softcap=25.0, window=40)
    k64, v64 = (x.double() for x in kv)
    pos = list(range(n + 3))
    want, tol = attention(q.double(), k64, v64, 0.09, torch.bfloat16, 2.0 ** -8,
                          first=[max(0, p - 39) for p in pos], last=pos, pos=pos, cap=25.0)
    cache.append([0], [n], kv[0][:n].cuda(), kv[1][:n].cuda())
    table, lens, longest = cache.tables([0], 12)
    got = cache.decode_multi(q[:n].cuda(), table, lens, torch.tensor([0, n], dtype=torch.int32).cuda(),
                             longest, n, 0.09, rule=rule)
    assert worst(got, want[:n], tol[:n]) <= 1
    step = torch.zeros(1, heads * group, dim, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(step)
    cache.decode(step, table, lens, 12 * bs, 0.09, out=out, rule=rule)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.decode(step, table, lens, 12 * bs, 0.09, out=out, rule=rule)
    for i in range(n, n + 3):
        cache.append([0], [1], kv[0][i:i + 1].cuda(), kv[1][i:i + 1].cuda())
        t, l, _ = cache.tables([0], 12)
        table.copy_(t)
        lens.copy_(l)
        step.copy_(q[i:i + 1])
        graph.replay()
        assert worst(out, want[i:i + 1], tol[i:i + 1]) <= 1
    with pytest.raises(ValueError):
        cache.decode(step, table, lens, 12 * bs, 0.09, rule=rule, groups=cache.groups(table, lens))
