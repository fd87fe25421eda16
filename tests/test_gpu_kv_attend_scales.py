"""Attention over the packed cache where the scales of neighbouring rows differ by what fp16 cannot
hold at once, and where rows that nobody may read hold anything. The bounds are those of
test_gpu_kv_attend.
"""

import numpy as np
import pytest
import torch

from test_gpu_kv_attend import Batch, check, queries, run

pytestmark = pytest.mark.gpu

# (queries of each sequence, query heads per key head): tiles of 16, 128 and 256 rows
TILES = [(1, 3), (40, 2), (150, 2)]


def scales_of(bt, part):
    """[pages, heads, page_tokens, groups] view of a half's scales."""
    return part.scales.view(-1, bt.heads, bt.page, bt.D // part.group)


def unused(bt, part):
    """Mask over the rows of a half that hold no token of any sequence."""
    free = torch.ones((part.E, bt.heads, bt.page), dtype=torch.bool)
    for slots in bt.slots:
        free[slots // bt.page, :, slots % bt.page] = False
    return free.cuda()


@pytest.mark.parametrize("n,share", TILES)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_that_hold_no_token_change_nothing(D, n, share):
    # 0.1 times the usual key scales: beside a scale of 65504 they would be held as fp16's subnormals
    lens = [n + 20, n + 67, n + 1]
    counts = [n] * 3
    bt = Batch(lens, heads=2, D=D, page=48, kg=32, seed=n)
    bt.cache.k.scales.mul_(0.1)
    bt.refresh()
    q = queries(3 * n, 2 * share, D, torch.bfloat16) * 20.0
    want = run(bt, q, counts)
    check(want, bt, q, counts, D ** -0.5, only={0, n - 1, n, 2 * n, 3 * n - 1})
    g = torch.Generator(device="cuda").manual_seed(D + n)
    for bits in (0x7bff, 0xfbff - 0x10000, 0x0001, 0x7c00, 0x7e00, None):
        for part in (bt.cache.k, bt.cache.v):
            free = unused(bt, part)
            s = scales_of(bt, part).view(torch.int16)
            any_bits = torch.randint(-0x8000, 0x8000, s.shape, generator=g, device="cuda", dtype=torch.int16)
            s[free] = any_bits[free] if bits is None else bits
            c = part.codes.view(*free.shape, -1)
            c[free] = torch.randint(-2 ** 31, 2 ** 31, c.shape, generator=g, device="cuda", dtype=torch.int64).to(torch.int32)[free]
        same = torch.equal(run(bt, q, counts), want)
        assert same, bits
