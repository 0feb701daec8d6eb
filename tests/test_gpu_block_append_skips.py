"""Skipped (negative) slots between the tokens of a block in the append to a
block-scaled E4M3 cache: bit-exact against the plain reference, which gathers a
block's tokens wherever they stand."""
import pytest
import torch

import paged_kv_cache_443_b200 as pk
from test_gpu_block_cache import Pool, draw

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_status():
    pk.pa_device_status(clear=True)
    yield
    torch.cuda.synchronize()
    assert pk.pa_device_status() == 0


def with_poison(x, slots):
    """Rows of skipped slots hold what would be the largest, or a NaN."""
    x = x.clone()
    skipped = torch.tensor([s < 0 for s in slots])
    x[skipped.cuda()] = 60000.0
    x[skipped.cuda(), :, ::3] = float("nan")
    return x


def check(pool, gen, slots, heads, dim, dtype, spread=3):
    n = len(slots)
    pool.append(*(with_poison(draw(gen, n, heads, dim, dtype, spread), slots) for _ in range(2)), slots)
    pool.check()


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("gap", [1, 2, 13, 14, 15, 16, 29, 30, 31, 32, 61, 62, 63, 190, 400])
def test_one_gap_inside_a_block(dtype, gap):
    """Two tokens of a block with `gap` skipped slots between them: beside another
    block's on either side, as the whole call, begun anew and not."""
    gen = torch.Generator().manual_seed(gap)
    pool = Pool(8, 2, 16, 128)
    for first in (0, 5):                                    # offset 0 begins the block anew
        two = lambda b: [b * 16 + first] + [-1] * gap + [b * 16 + first + 1]
        check(pool, gen, two(0), 2, 128, dtype)
        check(pool, gen, [-1] * 3 + two(1) + [-7] * gap, 2, 128, dtype)
        check(pool, gen, [32, 33] + two(3) + [4 * 16 + 3] + two(5), 2, 128, dtype, 6)


@pytest.mark.parametrize("dtype,dim,bs,heads,blocks", [
    (torch.bfloat16, 128, 16, 2, 40), (torch.float16, 64, 32, 3, 40), (torch.float32, 64, 8, 1, 60),
    (torch.bfloat16, 64, 16, 20, 250), (torch.float32, 128, 32, 8, 150), (torch.float16, 128, 8, 16, 400)])
@pytest.mark.parametrize("often", [2, 6, 25])
def test_gaps_anywhere(dtype, dim, bs, heads, blocks, often):
    """Runs of every length with skipped slots before, between and behind them; the
    larger calls have warps that look after up to 16 positions."""
    gen = torch.Generator().manual_seed(often * bs + blocks)
    pick = lambda *of: of[int(torch.randint(len(of), (1,), generator=gen))]
    pool = Pool(blocks, heads, bs, dim)
    for spread in (2, 5):
        slots = []
        for b in torch.randperm(blocks, generator=gen).tolist():
            n = min(bs, pick(1, 1, 2, 7, bs - 1, bs))
            for o in sorted(torch.randperm(bs, generator=gen)[:n].tolist()):
                if pick(*range(often)) == 0:
                    slots += [-1] * pick(1, 1, 2, 15, 16, 17, 33, 100)
                slots.append(b * bs + o)
        check(pool, gen, slots + [-1] * pick(0, 40, 300), heads, dim, dtype, spread)


def test_decode_steps_of_a_padded_batch():
    """One token a sequence, padding behind, between and in front."""
    gen = torch.Generator().manual_seed(3)
    pool = Pool(700, 8, 16, 128)
    for step, (front, behind) in enumerate([(0, 412), (300, 0), (1, 1), (0, 0)]):
        slots = [-1] * front
        for b in range(600):
            slots += [b * 16 + 3 + step] + [-1] * (b % 5 == step)
        check(pool, gen, slots + [-1] * behind, 8, 128, torch.bfloat16)


def test_a_long_stretch_of_skipped_slots():
    """Tokens of one block 20000 positions apart, and a run given one slot often."""
    gen = torch.Generator().manual_seed(4)
    pool = Pool(4, 1, 32, 64)
    check(pool, gen, [3] + [-1] * 20000 + [4, 40] + [-2] * 9000 + [41, 42], 1, 64, torch.float16)
    check(pool, gen, [64 + i // 2 if i % 2 else -1 for i in range(64)] + [-1] * 70 + [97], 1, 64,
          torch.float16)
