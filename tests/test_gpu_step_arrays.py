"""Where the arrays of a step's calls may lie, and where not."""

import numpy as np
import pytest
import torch

import rotation_lloyd_max_amd as tq
from test_gpu_verify import case, on_gpu, reference

pytestmark = pytest.mark.gpu


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_outputs_in_arrays_of_the_call_are_refused():
    pool, table = tq.kv_pool(8), torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    lens, counts = i32(0, 0), i32(20, 5)
    p = tq.kv_plan(pool, lens, counts, table, 25, 16)
    kept, before = i32(2, 1), [x.clone() for x in (pool.free, pool.state, table, *p[:5])]
    for more in (dict(out=kept), dict(out=p.status, status=p.status), dict(out=p.q_offsets[1:], q_offsets=p.q_offsets),
                 dict(out=table.view(-1)[1:3]), dict(out=pool.free[:2]), dict(out=pool.state), dict(left=kept[1:]),
                 dict(left=pool.state[1:]), dict(left=pool.free[7:]), dict(left=lens[:1])):
        with pytest.raises(tq.TqError, match="overlap"):
            tq.kv_keep(pool, lens, kept, table, 16, **more)
    for left in (pool.state[1:], lens[1:], table.view(-1)[3:4], counts[:1], pool.free[:1]):
        with pytest.raises(tq.TqError, match="overlap"):
            tq.kv_plan(pool, lens, counts, table, 25, 16, left=left)
    torch.cuda.synchronize()
    for a, b in zip(before, (pool.free, pool.state, table, *p[:5])):
        assert torch.equal(a, b)
    c = on_gpu(case(1, 3, 4, 100, ragged=False))
    with pytest.raises(tq.TqError, match="overlap"):
        tq.verify(**c, ws=c["target"])


def test_arrays_next_to_each_other_and_between_rows():
    # lens, counts, kept and the new lengths in one tensor; left taken as the pool's own count
    pool, table = tq.kv_pool(8), torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    whole = i32(0, 0, 20, 5, 2, 1, -7, -7, -9)
    p = tq.kv_plan(pool, whole[0:2], whole[2:4], table, 25, 16, left=pool.state[:1])
    assert pool.state.tolist() == [5, 0] and p.status.tolist() == [0, 0]
    tq.kv_keep(pool, whole[0:2], whole[4:6], table, 16, q_offsets=p.q_offsets, out=whole[6:8], left=whole[8:])
    assert whole.tolist() == [0, 0, 20, 5, 2, 1, 2, 1, 6] and pool.state.tolist() == [5, 0]
    # the outputs of verify behind the ends of the rows of its logits
    c = case(2, 3, 4, 100, "fp32", "fp32", ragged=False)
    g = on_gpu(c)
    M, V = 12, 100
    wide = torch.zeros((2, M, 128), device="cuda")
    for k, name in enumerate(("target", "draft")):
        wide[k, :, :V] = g[name]
    at = [wide.data_ptr() + 4 * (128 * r + V) for r in (0, 5, M + 3)]
    need = tq.verify_workspace(V, 3, M, True)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    rc = tq.lib().tq_verify(wide[0].data_ptr(), tq.F32, 128, wide[1].data_ptr(), tq.F32, 128, 0, V, 3, g["offsets"].data_ptr(), M,
                            g["tokens"].data_ptr(), None, g["uniforms"].data_ptr(), None, *at, ws.data_ptr(), need,
                            torch.cuda.current_stream().cuda_stream)
    assert rc == 0, tq.lib().tq_last_error()
    torch.cuda.synchronize()
    kept, tokens, path, _ = reference(c)
    flat = wide.view(-1).view(torch.int32)
    for want, n, r in ((kept, 3, 0), (tokens, M, 5), (path, M, M + 3)):
        assert np.array_equal(flat[128 * r + V:128 * r + V + n].cpu().numpy(), want)


@pytest.mark.parametrize("B,rows,vocab", [(1, 4, 32000), (8, 4, 20000), (16, 6, 131072), (64, 2, 131072)])
def test_what_the_results_of_verify_hold(B, rows, vocab):
    # programs keep them for many steps: of the workspace they hold 64 KiB at most
    M = B * rows
    t = torch.randn((M, vocab), dtype=torch.bfloat16, device="cuda")
    got = tq.verify(t, torch.zeros(M, dtype=torch.int32, device="cuda"), torch.rand(M, device="cuda"),
                    torch.arange(0, M + 1, rows, dtype=torch.int32, device="cuda"), draft=t)
    for x in got:
        assert x.untyped_storage().nbytes() <= 65536 + 4 * (B + 2 * M)
