"""PagedKVCache on a stream that is not the current one: every tensor that a call
makes by itself belongs to the launch's stream, or is known to be in use there
until its work is done (CPU only: streams and launches are recorded, not run)."""
import contextlib

import pytest
import torch

import paged_kv_cache_443_b200.cache as pc
from paged_kv_cache_443_b200 import BlockAllocator, Groups, ScoreRule
from paged_kv_cache_443_b200.cache import PagedKVCache

F8 = torch.float8_e4m3fn
LAUNCHES = [n for n in dir(pc) if n.startswith("pa_") and not n.endswith("_bytes")
            and n != "pa_build_groups"]


class Stream:
    def __init__(self, handle, device=None):
        self.cuda_stream = handle


@pytest.fixture
def gpu(monkeypatch):
    """Records the stream each tensor is made on, the streams it is marked as used
    on, and the tensors and the stream of each launch."""
    from paged_kv_cache_443_b200 import build
    build.build()
    rec = type("Record", (), {})()
    rec.stack, rec.born, rec.used, rec.launches, rec.keep = [Stream(0x10)], {}, {}, [], []

    @contextlib.contextmanager
    def on(stream):
        rec.stack.append(stream)
        yield
        rec.stack.pop()

    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: rec.stack[-1])
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream(0))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, s: rec.used.setdefault(id(t), []).append(s.cuda_stream))
    for name in ("empty", "empty_like", "tensor"):
        def make(*args, _real=getattr(torch, name), _name=name, **kw):
            t = _real(*args, **kw)
            rec.keep.append(t)
            rec.born[id(t)] = (rec.stack[-1].cuda_stream, _name)
            return t
        monkeypatch.setattr(torch, name, make)
    for name in LAUNCHES:
        def launch(*args, _name=name, stream=None, **kw):
            handle = rec.stack[-1].cuda_stream if stream is None else \
                getattr(stream, "cuda_stream", stream)
            made = [t for t in (*args, *kw.values()) if id(t) in rec.born]
            rec.launches.append((_name, handle, made))
        monkeypatch.setattr(pc, name, launch)
    return rec


def steps(cache, dtype, stream):
    """Every call of PagedKVCache that launches, with what it makes left to it."""
    x = torch.zeros(20, 2, 128, dtype=dtype)
    q = torch.zeros(2, 8, 128, dtype=dtype)
    cache.add(0)
    cache.append([0], [20], x, x, stream=stream)
    cache.fork(0, 1)
    cache.append([0, 1], [1, 1], x[:2], x[:2], stream=stream)       # copies the shared block
    table, lens, longest = cache.tables([0, 1])
    outs = []
    if not cache.fp8:
        rule = ScoreRule(softcap=30.0)
        start = torch.zeros(3, dtype=torch.int32)
        for r in (None, rule):
            outs.append(cache.decode_multi(q, table, lens, start, 4000, 1, 0.1, stream=stream, rule=r))
        outs.append(cache.decode(q, table, lens, 4000, 0.1, stream=stream, rule=rule))
    outs.append(cache.decode(q, table, lens, 4000, 0.1, stream=stream))
    if not cache.block_scales:
        groups = Groups(torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 1, 2, 16)
        outs.append(cache.decode(q, table, lens, 4000, 0.1, stream=stream, groups=groups))
    cache.swap_out([1], stream=stream)
    cache.swap_in([1], stream=stream)
    return outs


def make_cache(kind):
    dtype = torch.bfloat16 if kind == "bf16" else F8
    cache = PagedKVCache(40, 16, 2, 128, dtype, device="cpu", block_scales=kind == "block")
    cache.host_alloc = BlockAllocator(20, 16)          # enable_swap() without pinned memory
    cache.host_k = cache.host_v = cache.k_cache
    return cache


@pytest.mark.parametrize("kind", ["bf16", "fp8", "block"])
@pytest.mark.parametrize("given", ["stream", "handle", "default"])
def test_tensors_made_for_another_stream(gpu, kind, given):
    handle = {"stream": 0x20, "handle": 0x30, "default": 0}[given]
    cache = make_cache(kind)
    gpu.born.clear()
    outs = steps(cache, torch.bfloat16, Stream(handle) if given == "stream" else handle)
    assert len(gpu.launches) >= 6
    seen = set()
    for name, on, made in gpu.launches:
        assert on == handle
        for t in made:
            where, by = gpu.born[id(t)]
            if by == "tensor":     # uploaded: complete when it is returned, then read on `on`
                assert on == where or on in gpu.used.get(id(t), ()), name
            else:                  # written by the launch: no memory that another stream may still use
                assert on == where, name
            seen.add(by)
    assert seen == {"empty", "empty_like", "tensor"}
    for out in outs:               # the caller's from here on: freed after the current stream's work too
        assert 0x10 in gpu.used.get(id(out), ())


@pytest.mark.parametrize("given", [None, Stream(0x10), 0x10])
def test_the_current_stream_needs_none_of_it(gpu, given):
    gpu.born.clear()
    for kind in ("bf16", "block"):
        steps(make_cache(kind), torch.bfloat16, given)
    assert {on for _, on, _ in gpu.launches} == {0x10}
    assert not gpu.used and {w for w, _ in gpu.born.values()} == {0x10}


def test_the_legacy_default_stream_has_two_handles(gpu):
    gpu.stack[0] = Stream(0)
    for handle in (0, 1):
        steps(make_cache("bf16"), torch.bfloat16, handle)
    assert not gpu.used and {w for w, _ in gpu.born.values()} == {0}
