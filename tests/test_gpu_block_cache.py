"""The E4M3 cache with a scale per (block, kv head) on the GPU: append and copies
bit-exact against the plain reference, decode within the error its arithmetic
may leave (operators_ref), and the calls together through PagedKVCache."""
import numpy as np
import pytest
import torch

import paged_kv_cache_443_b200 as pk
from operators_ref import append, attention, e4m3_encode, gather, worst
from paged_kv_cache_443_b200.cache import PagedKVCache

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn
TYPES = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(autouse=True)
def clean_status():
    pk.pa_device_status(clear=True)
    yield
    torch.cuda.synchronize()
    assert pk.pa_device_status() == 0


class Pool:
    """A pool on the GPU and its reference, filled with NaN codes and NaN scales."""

    def __init__(self, blocks, heads, bs, dim):
        self.k, self.v = (torch.full((blocks, heads, bs, dim), 0x7f, dtype=torch.uint8, device="cuda")
                          for _ in range(2))
        self.ks, self.vs = (torch.full((blocks, heads), float("nan"), device="cuda") for _ in range(2))
        self.ref = [t.cpu().numpy().copy() for t in (self.k, self.v, self.ks, self.vs)]

    def tensors(self):
        return self.k.view(F8), self.v.view(F8), self.ks, self.vs

    def append(self, key, value, slots, ref=True):
        pk.pa_reshape_and_cache_fp8_block(key, value, *self.tensors(),
                                          torch.tensor(slots, dtype=torch.int64, device="cuda"))
        if ref:
            append(key.float().cpu().numpy(), self.ref[0], self.ref[2], slots)
            append(value.float().cpu().numpy(), self.ref[1], self.ref[3], slots)

    def check(self):
        for got, want in zip((self.k, self.v, self.ks, self.vs), self.ref):
            np.testing.assert_array_equal(got.cpu().numpy(), want)


def draw(gen, n, heads, dim, dtype, spread):
    x = torch.randn(n, heads, dim, generator=gen) * torch.exp2(
        torch.randint(-spread, spread + 1, (n, heads, 1), generator=gen).float())
    return x.to(dtype).cuda()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim,bs,heads", [(64, 8, 3), (64, 16, 1), (64, 32, 2), (128, 8, 2),
                                          (128, 16, 5), (128, 32, 1)])
def test_append_steps(dtype, dim, bs, heads):
    """Prompts, then many short calls: scales grow, older codes follow, padding."""
    gen = torch.Generator().manual_seed(dim + bs)
    alloc = pk.BlockAllocator(64, bs)
    pool = Pool(64, heads, bs, dim)
    for s, n in enumerate((1, bs - 1, bs, 2 * bs + 3)):
        alloc.add(s)
        slots, _ = alloc.append(s, n)
        pool.append(draw(gen, n, heads, dim, dtype, 2), draw(gen, n, heads, dim, dtype, 6), slots)
    pool.check()
    for step in range(12):
        slots = []
        for s in range(4):
            slots += alloc.append(s, (step + s) % 4)[0]
            slots += [-1] * (s == 2)
        if slots:
            pool.append(draw(gen, len(slots), heads, dim, dtype, 1 + step // 2),
                        draw(gen, len(slots), heads, dim, dtype, 5), slots)
    pool.check()


@pytest.mark.parametrize("dtype,heads,bs,n", [(torch.bfloat16, 8, 16, 2100), (torch.float32, 8, 32, 2100),
                                              (torch.float16, 20, 8, 900)])
def test_append_long_calls(dtype, heads, bs, n):
    """Calls long enough for warps that look after several positions, blocks whose
    runs straddle those, and as many one-token runs as positions."""
    gen = torch.Generator().manual_seed(n)
    pool = Pool(n // bs + 1200, heads, bs, 64)
    order = torch.randperm(n // bs + 1200, generator=gen).tolist()
    at = 5                                            # the first run starts inside a block
    slots = [order[(at + i) // bs] * bs + (at + i) % bs for i in range(n)]
    pool.append(draw(gen, n, heads, 64, dtype, 3), draw(gen, n, heads, 64, dtype, 3), slots)
    single = [b * bs + (b % bs) for b in order[-1100:]]
    pool.append(draw(gen, 1100, heads, 64, dtype, 3), draw(gen, 1100, heads, 64, dtype, 3), single)
    pool.check()


def test_append_special_values():
    """Zeros, NaN, infinities, the largest and smallest numbers, exact powers, and
    stored scales that are no powers of two, negative or NaN."""
    pool = Pool(16, 1, 8, 64)
    rows = torch.zeros(9, 1, 64)
    rows[1, 0, :4] = torch.tensor([448.0, -448.0, 1.0, -0.0])
    rows[2, 0, 3] = 448.0 * 2 ** -10 * (1 + 2 ** -23)          # just past a power
    rows[3, 0, :3] = torch.tensor([float("nan"), 1.5, -2.0])
    rows[4, 0, :3] = torch.tensor([float("inf"), float("-inf"), 3.0])
    rows[5, 0, :2] = torch.tensor([3.4e38, -1e30])
    rows[6, 0, :2] = torch.tensor([1e-40, -1e-38])
    rows[7, 0, :] = float("nan")
    rows[8, 0, 0] = 448.0 * 2.0 ** 80
    key = rows.cuda()
    pool.append(key, key.flip(0).contiguous(), [b * 8 for b in range(9)])
    # the next tokens of the same blocks, over changed stored scales
    stored = torch.tensor([1.0, 0.3, 5e-5, float("nan"), -1.0, 1e30, 0.0, 2.0, 0.7])
    for t, r in ((pool.ks, 2), (pool.vs, 3)):
        t[:9, 0] = stored.cuda()
        pool.ref[r][:9, 0] = stored.numpy()
    x = torch.linspace(-900, 900, 9 * 64).reshape(9, 1, 64).cuda()
    pool.append(x, x * 2.0 ** -12, [b * 8 + 1 + b % 7 for b in range(9)])
    pool.check()


def test_append_to_a_block_begun_anew_keeps_the_rest():
    """Offset 0 forgets the stored scale; unwritten slots keep their bytes."""
    pool = Pool(3, 2, 8, 64)
    gen = torch.Generator().manual_seed(4)
    pool.append(draw(gen, 8, 2, 64, torch.float16, 3), draw(gen, 8, 2, 64, torch.float16, 3),
                [8 + i for i in range(8)])
    pool.append(draw(gen, 3, 2, 64, torch.float16, 0) * 2 ** -9,
                draw(gen, 3, 2, 64, torch.float16, 0) * 2 ** -9, [9, 8, 12])
    pool.check()


def test_append_runs_longer_than_a_register_chunk():
    """A slot given several times in a row: the block's scale holds all of them, and
    the other slots of the call are right."""
    pool = Pool(2, 1, 32, 128)
    gen = torch.Generator().manual_seed(7)
    x = draw(gen, 70, 1, 128, torch.bfloat16, 2)
    slots = [31] * 40 + list(range(1, 31))
    pool.append(x, x, slots, ref=False)
    ref = [r.copy() for r in pool.ref]
    append(x.float().cpu().numpy(), ref[0], ref[2], slots)
    keep = list(range(31))
    np.testing.assert_array_equal(pool.ks.cpu().numpy(), ref[2])
    np.testing.assert_array_equal(pool.k.cpu().numpy()[:, :, keep], ref[0][:, :, keep])


def test_append_flags_slots_outside_the_pool():
    pool = Pool(2, 1, 8, 64)
    x = draw(torch.Generator().manual_seed(1), 4, 1, 64, torch.float16, 0)
    pool.append(x, x, [3, 16, -5, 1 << 40], ref=False)
    append(x.float().cpu().numpy(), pool.ref[0], pool.ref[2], [3, -1, -1, -1])
    append(x.float().cpu().numpy(), pool.ref[1], pool.ref[3], [3, -1, -1, -1])
    pool.check()
    assert pk.pa_device_status() == pk.PA_DEVERR_SLOT
    empty = x[:0]
    pool.append(empty, empty, [])
    pool.check()


@pytest.mark.parametrize("heads,dim,bs,pairs", [(1, 64, 8, 1), (5, 64, 32, 7), (40, 128, 16, 33),
                                                (8, 128, 32, 300)])
def test_copies(heads, dim, bs, pairs):
    gen = torch.Generator().manual_seed(pairs)
    pools = [Pool(2 * pairs + 3, heads, bs, dim) for _ in range(2)]
    for p in pools:
        for t, r in ((p.k, 0), (p.v, 1)):
            t.copy_(torch.randint(0, 256, t.shape, generator=gen, dtype=torch.uint8))
            p.ref[r] = t.cpu().numpy().copy()
        for t, r in ((p.ks, 2), (p.vs, 3)):
            t.copy_(torch.rand(t.shape, generator=gen))
            p.ref[r] = t.cpu().numpy().copy()
    order = torch.randperm(2 * pairs + 3, generator=gen)[:2 * pairs].reshape(pairs, 2)
    a, b = pools
    pk.pa_copy_blocks_fp8_block(*a.tensors(), order.cuda())
    for r in a.ref:
        r[order[:, 1].numpy()] = r[order[:, 0].numpy()]
    a.check()
    pk.pa_swap_blocks_fp8_block(*b.tensors(), *a.tensors(), order.cuda())
    for r, s in zip(b.ref, a.ref):
        r[order[:, 1].numpy()] = s[order[:, 0].numpy()]
    b.check()
    pk.pa_copy_blocks_fp8_block(*a.tensors(), order[:0].cuda())
    a.check()
    pk.pa_copy_blocks_fp8_block(*a.tensors(), torch.tensor([[0, 2 * pairs + 3], [-1, 1]]).cuda())
    a.check()
    assert pk.pa_device_status() == pk.PA_DEVERR_PAIR


def test_swap_with_pinned_memory():
    a = Pool(6, 3, 16, 128)
    gen = torch.Generator().manual_seed(3)
    x = draw(gen, 96, 3, 128, torch.bfloat16, 3)
    a.append(x, x, list(range(96)))
    host = [torch.zeros(t.shape, dtype=t.dtype).pin_memory() for t in (a.k, a.v, a.ks, a.vs)]
    view = (host[0].view(F8), host[1].view(F8), host[2], host[3])
    pk.pa_swap_blocks_fp8_block(*view, *a.tensors(), torch.tensor([[0, 5], [4, 1]]).cuda())
    torch.cuda.synchronize()
    for h, r in zip(host, a.ref):
        np.testing.assert_array_equal(h.numpy()[[5, 1]], r[[0, 4]])
        assert not h.numpy()[[0, 2, 3, 4]].any()
    pk.pa_swap_blocks_fp8_block(*a.tensors(), *view, torch.tensor([[1, 0]]).cuda())
    for r in a.ref:
        r[0] = r[4]
    a.check()


# ---- decode ----


def random_pool(gen, blocks, heads, bs, dim, low, high):
    """Codes and scales 2^low .. 2^high on the CPU."""
    codes = e4m3_encode((torch.randn(blocks, heads, bs, dim, generator=gen) * 90).numpy())
    scales = torch.exp2(torch.randint(low, high + 1, (blocks, heads), generator=gen).float())
    return torch.from_numpy(codes), scales


class Batch:
    """Sequences over a block-scaled cache; unused slots hold NaN codes, unused
    blocks NaN scales."""

    def __init__(self, gen, lens, heads, bs, dim, k_range=(-9, -5), v_range=(-9, -3)):
        need = [-(-n // bs) for n in lens]
        self.blocks = sum(need) + 3
        self.k, self.ks = random_pool(gen, self.blocks, heads, bs, dim, *k_range)
        self.v, self.vs = random_pool(gen, self.blocks, heads, bs, dim, *v_range)
        self.lens, self.bs, self.dim, self.heads = list(lens), bs, dim, heads
        order = torch.randperm(self.blocks, generator=gen).int()
        self.table = torch.full((len(lens), max(need) + 1), -1, dtype=torch.int32)
        for b, n in enumerate(need):
            self.table[b, :n] = order[sum(need[:b]):sum(need[:b]) + n]
            if lens[b] % bs:
                for t in (self.k, self.v):
                    t[self.table[b, n - 1].long(), :, lens[b] % bs:] = 0x7f
        for t in (self.ks, self.vs):
            t[order[sum(need):].long()] = float("nan")

    def run(self, q, scale, partition=0, workspace_fill=True):
        dev = [t.cuda() for t in (self.k, self.v, self.ks, self.vs, self.table)]
        lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        out = torch.full_like(q, float("nan")).cuda()
        n = pk.pa_decode_workspace_bytes(len(self.lens), q.shape[1], self.dim, max(self.lens), partition)
        ws = torch.full((n // 4,), float("nan"), device="cuda") if n else None
        pk.pa_decode_fp8_block(out, q.cuda(), dev[0].view(F8), dev[1].view(F8), dev[2], dev[3],
                               dev[4], lens, scale, max(self.lens), partition_size=partition,
                               workspace=ws)
        return out

    def want(self, q, scale):
        G = q.shape[1] // self.heads
        # both 16-bit types may run on the tensor cores at head size 128: P is then
        # held to 2^-8 (two E4M3 terms) for bf16 and 2^-12 (three) for f16 queries,
        # which on the CUDA cores (short contexts at one head; head size 64 at up to
        # two) have it in f16; else it is fp32
        tensor_core = self.dim == 128 and q.dtype != torch.float32
        u_p = 0.0
        if q.dtype == torch.float16 and (tensor_core or G <= 2):
            u_p = 2.0 ** -11
        elif tensor_core:
            u_p = 2.0 ** -8
        out, tol = [], []
        for b, n in enumerate(self.lens):
            if n == 0:
                out.append(torch.zeros(1, *q.shape[1:], dtype=torch.float64))
                tol.append(torch.zeros_like(out[-1]))
                continue
            k, _ = gather(self.k, self.table[b], n, self.ks)
            v, vs = gather(self.v, self.table[b], n, self.vs)
            o, t = attention(q[b:b + 1].double(), k, v, scale, q.dtype, u_p, split=tensor_core,
                             floor_values=vs)
            out.append(o)
            tol.append(t)
        return torch.cat(out), torch.cat(tol)

    def check(self, q, scale, partition=0):
        got = self.run(q, scale, partition).cpu().double()
        out, tol = self.want(q, scale)
        assert worst(got, out, tol) <= 1
        return got


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group,heads,bs", [(1, 3, 8), (2, 2, 16), (4, 2, 32), (8, 1, 8), (8, 2, 16)])
def test_decode(dtype, dim, group, heads, bs):
    """Lengths around blocks, stages, tiles and partitions."""
    gen = torch.Generator().manual_seed(dim + group)
    lens = [0, 1, bs - 1, bs, bs + 1, 31, 33, 127, 128, 129, 255, 257, 511, 513, 700]
    batch = Batch(gen, lens, heads, bs, dim)
    q = torch.randn(len(lens), group * heads, dim, generator=gen).to(dtype)
    for partition in (0, 128, 256):
        batch.check(q, dim ** -0.5, partition)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("group", [1, 2, 4, 8])
def test_decode_scales_far_apart(dtype, group):
    """Value scales over 24 powers of two, all-zero blocks whose scale is 0, and
    scales that are no powers of two."""
    gen = torch.Generator().manual_seed(group)
    batch = Batch(gen, [900, 77, 300], 2, 16, 128, k_range=(-12, -6), v_range=(-20, 4))
    batch.ks = batch.ks * (0.75 + 0.5 * torch.rand(batch.ks.shape, generator=gen))
    batch.vs = batch.vs * (0.75 + 0.5 * torch.rand(batch.vs.shape, generator=gen))
    zero = batch.table[0, 3:9].long()
    batch.k[zero], batch.v[zero] = 0, 0
    batch.ks[zero], batch.vs[zero] = 0.0, 0.0
    q = torch.randn(3, 2 * group, 128, generator=gen).to(dtype)
    batch.check(q, 128 ** -0.5)
    batch.check(q, 128 ** -0.5, 128)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("group", [1, 2, 4, 8])
@pytest.mark.parametrize("over", [7.0, 9.7])
def test_decode_one_key_over_many(dtype, group, over):
    """A key that outweighs each of 6000 others by e^7 (e^9.7 = 2^14), which together
    weigh as much: small weights must not be lost, whatever the blocks' scales."""
    gen = torch.Generator().manual_seed(group)
    batch = Batch(gen, [6001], 1, 16, 128, v_range=(-7, -6))
    q = torch.sign(torch.randn(1, group, 128, generator=gen))
    q[:] = q[:, :1]
    one = e4m3_encode((q[0, 0] * 64).numpy())
    batch.k[batch.table[0, :376].long()] = 0
    batch.k[batch.table[0, 0].long(), 0, 0] = torch.from_numpy(one)
    batch.ks[:] = 1.0
    batch.v[batch.table[0, :376].long()] &= 0x7f      # positive values: no cancellation
    scale = over / (64 * 128)
    got = batch.check(q.to(dtype), scale)
    out, _ = batch.want(q.to(dtype), scale)
    # far inside the worst case: the mean of the weights' rounding errors
    assert float(((got - out).abs() / out.abs()).max()) < 2.0 ** -7


def test_decode_agrees_with_the_cache_of_one_scale():
    """With every block's scale the same power of two, the result of pa_decode_fp8."""
    gen = torch.Generator().manual_seed(5)
    batch = Batch(gen, [300, 1, 1000], 2, 16, 128)
    batch.ks[:], batch.vs[:] = 2.0 ** -6, 2.0 ** -5
    q = torch.randn(3, 8, 128, generator=gen).to(torch.bfloat16)
    got = batch.run(q, 0.09)
    out = torch.empty_like(got)
    ws = torch.empty(pk.pa_decode_workspace_bytes(3, 8, 128, 1000) // 4, device="cuda")
    pk.pa_decode_fp8(out, q.cuda(), batch.k.cuda().view(F8), batch.v.cuda().view(F8),
                     batch.table.cuda(), torch.tensor(batch.lens, dtype=torch.int32).cuda(), 0.09,
                     1000, 2.0 ** -6, 2.0 ** -5, workspace=ws)
    _, tol = batch.want(q, 0.09)
    assert worst(got, out.cpu().double(), 2 * tol) <= 1


@pytest.mark.parametrize("group", [1, 8])
def test_decode_flags_bad_blocks_and_lengths(group):
    gen = torch.Generator().manual_seed(2)
    batch = Batch(gen, [300, 40], 1, 16, 128)
    q = torch.randn(2, group, 128, generator=gen).to(torch.float16)
    want, tol = batch.want(q, 0.09)
    batch.table[0, 7] = batch.blocks
    batch.table[0, 9] = -3
    got = batch.run(q, 0.09).cpu().double()
    assert worst(got[1], want[1], tol[1]) <= 1
    assert pk.pa_device_status() == pk.PA_DEVERR_TABLE
    batch.lens[0] = -4
    batch.run(q, 0.09)
    assert pk.pa_device_status() == pk.PA_DEVERR_CONTEXT


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("group", [1, 2, 4, 8])
def test_decode_long_and_repeated(dtype, group):
    """Contexts over 1024 tokens (the tensor cores at every group size), many CTAs,
    partial last tiles: right, and every launch gives the same bytes."""
    gen = torch.Generator().manual_seed(8)
    lens = [int(x) for x in torch.randint(1, 1200, (64,), generator=gen)] + [1025, 2000]
    batch = Batch(gen, lens, 2, 16, 128)
    q = torch.randn(66, 2 * group, 128, generator=gen).to(dtype)
    batch.check(q, 0.09)
    batch.check(q, 0.09, 128)
    one = batch.run(q, 0.09)
    for _ in range(12):
        assert torch.equal(batch.run(q, 0.09), one)


# ---- together ----


@pytest.mark.parametrize("dtype,group", [(torch.bfloat16, 4), (torch.float16, 1)])
def test_cache_serves_forks_and_swaps(dtype, group):
    """PagedKVCache with block scales: prompt, forks that diverge (copy-on-write),
    decode, swap out and in; against a private history of every sequence."""
    gen = torch.Generator().manual_seed(11)
    heads, dim, bs = 2, 128, 16
    cache = PagedKVCache(64, bs, heads, dim, F8, block_scales=True)
    cache.enable_swap(64)
    ref = {n: r for n, r in zip(("k", "v", "ks", "vs"), (
        np.zeros((64, heads, bs, dim), np.uint8), np.zeros((64, heads, bs, dim), np.uint8),
        np.zeros((64, heads), np.float32), np.zeros((64, heads), np.float32)))}

    def store(seqs, counts, spread):
        n = sum(counts)
        key, value = draw(gen, n, heads, dim, dtype, spread), draw(gen, n, heads, dim, dtype, spread)
        slots, pairs = cache.append(seqs, counts, key, value)
        for src, dst in pairs:
            for r in ref.values():
                r[dst] = r[src]
        append(key.float().cpu().numpy(), ref["k"], ref["ks"], slots)
        append(value.float().cpu().numpy(), ref["v"], ref["vs"], slots)

    def check(seqs):
        table, lens, longest = cache.tables(seqs)
        q = torch.randn(len(seqs), heads * group, dim, generator=gen).to(dtype)
        got = cache.decode(q.cuda(), table, lens, longest, dim ** -0.5).cpu().double()
        for b in range(len(seqs)):
            n = int(lens[b])
            k, _ = gather(torch.from_numpy(ref["k"]), table[b].cpu(), n, torch.from_numpy(ref["ks"]))
            v, vs = gather(torch.from_numpy(ref["v"]), table[b].cpu(), n, torch.from_numpy(ref["vs"]))
            out, tol = attention(q[b:b + 1].double(), k, v, dim ** -0.5, dtype,
                                 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -11, split=True,
                                 floor_values=vs)
            assert worst(got[b], out[0], tol[0]) <= 1

    cache.add(0)
    store([0], [37], 1)
    for child in (1, 2):
        cache.fork(0, child)
    store([0, 1, 2], [1, 1, 3], 4)       # two copies, each then rescaled on its own
    check([0, 1, 2])
    before = {s: cache.tables([s])[0] for s in (1, 2)}
    for src, dst in cache.swap_out([1, 2]):
        pass
    cache.add(7)
    store([7], [100], 2)                 # takes the released blocks
    check([0, 7])
    moved = {}
    for seq in (1, 2):                   # the reference follows the moved blocks
        moved[seq] = [{n: r[b].copy() for n, r in ref.items()}
                      for b in before[seq][0].tolist() if b >= 0]
    back = cache.swap_in([1, 2])
    assert back
    k, v, ks, vs = (t.cpu() for t in (cache.k_cache.view(torch.uint8), cache.v_cache.view(torch.uint8),
                                      cache.k_scales, cache.v_scales))
    host = [cache.host_k.view(torch.uint8), cache.host_v.view(torch.uint8), cache.host_k_scales,
            cache.host_v_scales]
    for src, dst in back:
        for t, h, n in zip((k, v, ks, vs), host, ("k", "v", "ks", "vs")):
            assert torch.equal(t[dst], h[src])
            ref[n][dst] = h[src].numpy()
    check([0, 1, 7, 2])


def test_captured_step_and_two_streams():
    """Append and decode captured into one graph and replayed on new inputs, next
    to an eager stream that uses another pool and workspace."""
    gen = torch.Generator().manual_seed(13)
    batch = Batch(gen, [500, 129, 40], 2, 16, 128)
    dev = [t.cuda() for t in (batch.k, batch.v, batch.ks, batch.vs)]
    start = [t.clone() for t in dev]
    table = batch.table.cuda()
    lens = torch.tensor(batch.lens, dtype=torch.int32).cuda()
    n = pk.pa_decode_workspace_bytes(3, 8, 128, 500)
    ws = torch.empty(max(4, n // 4), device="cuda")
    q = torch.zeros(3, 8, 128, dtype=torch.bfloat16, device="cuda")
    key, value = (torch.zeros(3, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    at = [n - 1 for n in batch.lens]          # the newest token is written again
    slots = torch.tensor([int(batch.table[b, p // 16]) * 16 + p % 16 for b, p in enumerate(at)])
    slots = slots.cuda()
    out = torch.empty_like(q)

    def step(stream=None):
        pk.pa_reshape_and_cache_fp8_block(key, value, dev[0].view(F8), dev[1].view(F8), dev[2],
                                          dev[3], slots, stream=stream)
        pk.pa_decode_fp8_block(out, q, dev[0].view(F8), dev[1].view(F8), dev[2], dev[3], table, lens,
                               0.09, 500, partition_size=128, workspace=ws2, stream=stream)

    ws2 = torch.empty(pk.pa_decode_workspace_bytes(3, 8, 128, 500, 128) // 4, device="cuda")
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    other = torch.cuda.Stream()
    eager = Batch(gen, [333, 64], 1, 16, 128)
    eq = torch.randn(2, 4, 128, generator=gen).to(torch.bfloat16)
    want_e, tol_e = eager.want(eq, 0.09)
    for trial in range(4):
        for t, s in zip(dev, start):
            t.copy_(s)
        q.copy_(torch.randn(q.shape, generator=gen))
        key.copy_(torch.randn(key.shape, generator=gen) * 2.0 ** (trial * 3))
        value.copy_(torch.randn(key.shape, generator=gen))
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(other):
            got_e = eager.run(eq, 0.09)
        torch.cuda.synchronize()
        assert worst(got_e, want_e, tol_e) <= 1
        ref = [s.cpu().numpy().copy() for s in start]
        append(key.float().cpu().numpy(), ref[0], ref[2], slots.tolist())
        append(value.float().cpu().numpy(), ref[1], ref[3], slots.tolist())
        for t, r in zip(dev, ref):
            np.testing.assert_array_equal(t.cpu().numpy(), r)
        batch.k, batch.v, batch.ks, batch.vs = (torch.from_numpy(r) for r in ref)
        want, tol = batch.want(q.cpu(), 0.09)
        assert worst(out, want, tol) <= 1
