"""Rotary positions of more tokens than one launch holds: 2^24 + 5 tokens of a workgroup each (17 GB of
output) have more threads than 2^32. Every row against the same turn in small calls."""

import pytest
import torch

import rotation_lloyd_max_amd as tq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("transposed", [False, True])
def test_more_tokens_than_a_launch_holds(transposed):
    n, d = (1 << 24) + 5, 512
    r = tq.rope_frequencies(d)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((1, 1, d), generator=g, device="cuda").to(torch.bfloat16)
    # positions repeat every 4096 tokens, so that one small call has every row
    small = tq.rope(x.expand(4096, 1, d), torch.arange(4096, device="cuda"), r, transposed=transposed)
    pos = (torch.arange(n, device="cuda") % 4096).to(torch.int32)
    out = torch.zeros((n, 1, d), dtype=torch.bfloat16, device="cuda")
    tq.rope(x.expand(n, 1, d), pos, r, transposed=transposed, out=out)
    whole = out[:(1 << 24)].view(-1, 4096, 1, d)
    step = 256
    assert all(bool((whole[i:i + step] == small).all()) for i in range(0, whole.shape[0], step))
    assert torch.equal(out[1 << 24:], small[:5])
