"""Attention over the packed cache with many query rows per key head (chunks and trees), where
the waves split the rows: values of any size, rows that are no numbers, bad pages, masks, graphs.
The bounds are those of test_gpu_kv_attend.
"""

import numpy as np
import pytest
import torch

import rotation_lloyd_max_amd as tq
from test_gpu_kv_attend import Batch, check, queries, run, tree_rows

pytestmark = pytest.mark.gpu

# (counts, share): rows per key head and sequence on average 60 (a tile of 128) and 300 (of 256)
SIZES = [([30], 2), ([150], 2)]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("counts,share", SIZES)
@pytest.mark.parametrize("spread", [1e-4, 1.0, 3e3])
def test_values_of_any_size(spread, counts, share, D):
    # scales from fp16's subnormals to near its largest value, growing, shrinking and alternating
    # along the sequence: the powers of two change from block to block
    n = 333
    for shape in (lambda m: np.geomspace(spread * 0.01, spread * 10, m), lambda m: np.geomspace(spread * 10, spread * 0.01, m),
                  lambda m: spread * np.where(np.arange(m) // 32 % 2, 10.0, 0.01)):
        bt = Batch([n], heads=1, D=D, page=48, vl=256, dt=torch.float32, vscale=shape)
        q = queries(sum(counts), share, D, torch.bfloat16)
        check(run(bt, q, counts), bt, q, counts, D ** -0.5, only=set(range(0, sum(counts), 13)) | {sum(counts) - 1})


@pytest.mark.parametrize("counts,share", SIZES)
def test_keys_of_any_size(counts, share):
    # key scales 2^-13 and 2^14 times the usual, queries as much larger and smaller
    for f in (2.0 ** -13, 2.0 ** 14):
        bt = Batch([200], heads=1, D=128, page=16, kg=64)
        bt.cache.k.scales.mul_(f)
        bt.refresh()
        q = queries(sum(counts), share, 128, torch.bfloat16) * (1 / f)
        check(run(bt, q, counts), bt, q, counts, 128 ** -0.5, only=set(range(0, sum(counts), 13)))


@pytest.mark.parametrize("counts,share", SIZES)
@pytest.mark.parametrize("bits", [0x7e00, 0x7c00])
def test_rows_that_are_no_numbers_reach_their_readers_alone(counts, share, bits):
    n = counts[0]
    bt = Batch([n + 40, 64], heads=1, D=64, page=16, kg=32)
    q = queries(n + 40, share, 64, torch.bfloat16)
    both = [n, 40]
    want = run(bt, q, both)
    check(want, bt, q, both, 0.125, only={0, 7, n - 1, n + 39})
    j = 40 + n - 3                                  # seen by the last three queries of sequence 0
    for part in (bt.cache.k, bt.cache.v):
        keep = part.scales.clone()
        s = int(bt.slots[0][j])
        part.scales.view(torch.int16).view(-1, 1, 16, 2)[s // 16, :, s % 16] = bits
        got = run(bt, q, both)
        assert torch.equal(got[:n - 3], want[:n - 3]) and torch.equal(got[n:], want[n:])
        if bits == 0x7e00 or part is bt.cache.v:    # (an infinite key's scores may all be -inf)
            assert torch.isnan(got[n - 3:n]).all()
        part.scales.copy_(keep)
    # unused rows of the last pages may hold anything
    for part in (bt.cache.k, bt.cache.v):
        keep = part.scales.clone()
        part.scales.view(torch.int16).fill_(bits)
        for b in range(2):
            for s in bt.slots[b]:
                part.scales.view(-1, 1, 16, 2)[s // 16, :, s % 16] = keep.view(-1, 1, 16, 2)[s // 16, :, s % 16]
    assert torch.equal(run(bt, q, both), want)


@pytest.mark.parametrize("counts,share", SIZES)
def test_bad_pages_poison_their_readers_alone(counts, share):
    n = counts[0]
    bt = Batch([n + 70, 100], heads=2, D=128, page=16, kg=32)
    q = queries(n + 40, 2 * share, 128, torch.bfloat16)
    want = run(bt, q, [n, 40])
    at = (n + 70 - 1) // 16                         # the last page of sequence 0: from token 16 at on
    first = 16 * at - 70                            # first query that sees it
    for bad in (-1, bt.cache.k.E, 2 ** 31 - 1, -2 ** 31):
        table = bt.table.copy()
        bt.table[0, at] = bad
        got = run(bt, q, [n, 40])
        bt.table[:] = table
        assert torch.isnan(got[first:n]).all()
        assert torch.equal(got[:first], want[:first]) and torch.equal(got[n:], want[n:])


@pytest.mark.parametrize("j", [0, 31, 32, 63, 64, 159, 160, 161, 191, 192, 223])
def test_one_loud_token_is_seen_by_its_successors_alone(j):
    # the mask moved by one token anywhere would show a thousandfold
    bt = Batch([224], heads=1, D=64, page=16, kg=32)
    s = int(bt.slots[0][j])
    bt.cache.v.scales.view(-1, 1, 16, 2)[s // 16, :, s % 16] *= 1000.0
    bt.refresh()
    counts = [64]
    q = queries(64, 2, 64, torch.bfloat16)
    got = run(bt, q, counts)
    check(got, bt, q, counts, 0.125, only=set(range(0, 64, 9)) | {max(0, j - 160), max(0, j - 161), 63})
    # a mean of the values it sees is no longer than the longest of them (1.02: the roundings)
    longest = 1.02 * float(np.delete(np.linalg.norm(bt.rows[1][0][:, 0], axis=1), j).max())
    size = got.float().norm(dim=-1).amax(-1)
    assert all(j <= 160 + i or float(size[i]) <= longest for i in range(64))


def test_trees_that_leave_nothing_and_bits_past_the_words():
    counts, lens = [50, 30], [50, 30]
    bt = Batch(lens, heads=1, D=64, page=16, kg=32)
    tree = np.zeros((80, 32), dtype=np.uint8)
    tree[5, 2] = 1
    tree[39, :] = 1
    tree[51, 1] = 1
    q = queries(80, 2, 64, torch.bfloat16)
    got = run(bt, q, counts, tree)
    check(got, bt, q, counts, 0.125, tree)
    assert not got[0].any() and got[5].any() and got[39].any()


@pytest.mark.parametrize("qsize,scale", [(0.0, 0.1), (1e-6, 0.1), (300.0, 0.1), (1.0, 0.0), (1.0, -0.2)])
def test_queries_and_scales_of_any_size(qsize, scale):
    bt = Batch([300, 130], heads=1, D=64, page=16, kg=32)
    counts = [130, 130]
    q = queries(260, 3, 64, torch.bfloat16) * qsize
    check(run(bt, q, counts, scale=scale), bt, q, counts, scale, only=set(range(0, 260, 17)) | {259})


def test_strides_output_types_rows_behind_and_no_offsets():
    bt = Batch([150, 260], heads=2, D=128, page=16)
    wide = queries(70, 12, 128, torch.bfloat16)
    q = wide[:, :4]             # a slice of a fused projection
    want = run(bt, q.contiguous(), [30, 40])
    out = torch.full((70, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lens, table = bt.dev()
    off = torch.tensor([0, 30, 60], dtype=torch.int32, device="cuda")
    tq.kv_attend(bt.cache, q, lens, table, q_offsets=off, out=out)
    torch.cuda.synchronize()
    assert torch.equal(run(bt, q, [30, 40]), want) and torch.equal(out[:30], want[:30]) and torch.all(out[60:] == 7.0)
    half = run(bt, q, [30, 40], out_dtype=torch.float16)
    check(half, bt, q, [30, 40], 128 ** -0.5, only=set(range(0, 70, 11)))
    assert torch.equal(run(bt, q), run(bt, q, [35, 35]))


def test_chunks_beside_single_tokens():
    # one prompt among decoded tokens: rows of very different number in one call
    counts, lens = [1, 1, 200, 1, 0, 3, 1], [700, 1, 333, 90, 50, 64, 2000]
    bt = Batch(lens, heads=2, D=128, page=32)
    q = queries(sum(counts), 8, 128, torch.bfloat16)
    check(run(bt, q, counts), bt, q, counts, 128 ** -0.5, only={0, 1, 2, 3, 63, 64, 65, 129, 200, 201, 202, 203, 204, 205, 206})


def test_captured_chunks_replayed():
    bt = Batch([900, 260], heads=2, D=128, page=64)
    counts = [150, 60]
    g = np.random.default_rng(5)
    tree = tree_rows(counts, g, 160)
    words = torch.from_numpy(np.packbits(tree, axis=1, bitorder="little").view(np.int32).copy()).cuda()
    lens, table = bt.dev()
    off = torch.tensor([0, 150, 210], dtype=torch.int32, device="cuda")
    q = queries(210, 8, 128, torch.bfloat16)
    ws = torch.empty(tq.kv_attend_workspace(bt.cache, 8, 2, 210), dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(q) for _ in range(2)]
    graphs = []
    for o, t in zip(outs, (None, words)):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            tq.kv_attend(bt.cache, q, lens, table, q_offsets=off, tree=t, out=o, ws=ws)
        graphs.append(gr)
    for rep in range(4):
        q.copy_(queries(210, 8, 128, torch.bfloat16, seed=rep))
        ws.fill_(255)
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for o, t in zip(outs, (None, words)):
            assert torch.equal(o, tq.kv_attend(bt.cache, q, lens, table, q_offsets=off, tree=t)), rep
            o.zero_()


@pytest.mark.parametrize("n", [1, 40])
def test_sequences_on_the_same_pages(n):
    # a shared text: the same pages in several sequences' tables, and one page twice in a row of it
    bt = Batch([160, 160, 96], heads=2, D=64, page=32, kg=32)
    table = np.array(bt.table)
    table[1] = table[0]
    table[2, 2] = table[2, 0]
    bt.table[:] = table
    for b, m in ((1, 160), (2, 96)):
        j = np.arange(m)
        bt.slots[b] = table[b, j // 32].astype(np.int64) * 32 + j % 32
    bt.refresh()
    counts = [n, n, n]
    q = queries(3 * n, 4, 64, torch.bfloat16)
    q[n:2 * n] = q[:n]
    got = run(bt, q, counts)
    check(got, bt, q, counts, 0.125, only=set(range(0, 3 * n, 7)) | {3 * n - 1})
    want = got[:n] if n > 1 else got[:1]
    assert torch.allclose(got[n:2 * n].float(), want.float(), rtol=2.0 ** -6, atol=2.0 ** -6)


def test_two_streams_with_their_own_workspaces():
    bt = Batch([900, 260], heads=2, D=128, page=64)
    counts = [150, 60]
    off = torch.tensor([0, 150, 210], dtype=torch.int32, device="cuda")
    qs = [queries(210, 8, 128, torch.bfloat16, seed=s) for s in range(2)]
    want = [run(bt, q, counts) for q in qs]
    lens, table = bt.dev()
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in qs], [[], []]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(tq.kv_attend(bt.cache, qs[i], lens, table, q_offsets=off))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])
