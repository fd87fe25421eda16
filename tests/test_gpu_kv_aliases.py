"""Outputs that are, or lie beside, a call's inputs: attention into its own queries, rotary turns into a
neighbouring slice of the same buffer."""

import numpy as np
import pytest
import torch

import rotation_lloyd_max_amd as tq
from test_gpu_kv_attend import Batch, queries, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,counts,share", [([3000], [1], 4), ([70, 900, 33], [2, 5, 1], 3), ([700, 900], [40, 40], 2),
                                               ([5000, 300], [150, 150], 2), ([60] * 200, [1] * 200, 2)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_into_its_own_queries(D, lens, counts, share):
    bt = Batch(lens, heads=2, D=D, page=16)
    q = queries(sum(counts) + 2, 2 * share, D, torch.bfloat16)
    want = torch.cat([run(bt, q, counts)[:sum(counts)], q[sum(counts):]])
    assert torch.equal(run(bt, q, counts, out=q), want)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_rope_into_a_neighbouring_slice(dt):
    g = np.random.default_rng(3)
    wide = torch.from_numpy(g.standard_normal((37, 12, 64)).astype(np.float32)).cuda().to(dt)
    pos = torch.arange(37, dtype=torch.int32, device="cuda")
    r = tq.rope_frequencies(48)
    want = wide.clone()
    want[:, 6:10] = tq.rope(wide[:, 2:6].clone(), pos, r)
    tq.rope(wide[:, 2:6], pos, r, out=wide[:, 6:10])
    assert torch.equal(wide, want)


def test_wide_index_values_do_not_wrap():
    # 64-bit pages and lengths: 2^32 + p is no page p, 2^32 + 16 is a length beyond the table
    bt = Batch([40, 48], heads=1, D=64, page=16, kg=32)
    q = queries(2, 2, 64, torch.bfloat16)
    lens, table = (t.to(torch.int64) for t in bt.dev())
    want = run(bt, q)
    assert torch.equal(tq.kv_attend(bt.cache, q, lens, table), want)
    bad = table.clone()
    bad[0, 1] += 2 ** 32
    got = tq.kv_attend(bt.cache, q, lens, bad)
    assert torch.isnan(got[0]).all() and torch.equal(got[1], want[1])
    far = lens.clone()
    far[1] = 2 ** 32 + 16
    assert torch.equal(tq.kv_attend(bt.cache, q, far, table), want)
