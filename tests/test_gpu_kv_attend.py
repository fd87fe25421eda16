"""Attention over the packed cache against the oracle: dequantized, rotated back and attended in
fp64, from the codes that the GPU stored.

Bound per query row and head, in the 2-norm (the rotations keep it), with u = 2^-11, half a step
of fp16, the type of the matrix cores' operands:
  scores    rotated q, the key's centroid and its product with the scale rounded to fp16, fp32
            sums: |ds_j| <= E_j = |scale| ((3 u + (D + 16) 2^-24) sum_d |q'_d k'_jd| +
            2^-19 max|q'| sum_d |k'_jd|) + 2^-21 |s_j|
            (the last terms: the fp32 transform of q and the exponent's argument)
  weights   p_j off by a factor within e^(2 max E), and u + 2^-19 from the rounding of p and exp
  values    the centroid and its product with the scale rounded to fp16: 2 u
  sums      n 2^-24 of the sum of |terms|
so |do'_d| <= (expm1(2 max E) + 3 u + 2^-18 + n 2^-24) sum_j p_j |v'_jd|, and one rounding of out.
"""

import numpy as np
import pytest
import torch

import rotation_lloyd_max_amd as tq
from oracle import attention as oat
from oracle import encode as oenc
from oracle import hadamard as ohd
from parity import as_f64, torch_to_np

pytestmark = pytest.mark.gpu
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
U = 2.0 ** -11


class Batch:
    """Sequences of `lens` tokens in shuffled pages of a cache that kv_store filled."""

    def __init__(self, lens, heads, D, page, kl=256, vl=8, kg=64, vg=None, seed=0, dt=torch.bfloat16, spare=1,
                 vscale=None):
        g = np.random.default_rng([seed, D, len(lens)])
        need = [-(-n // page) for n in lens]
        pages = sum(need) + spare
        self.cache = tq.kv_cache(pages, heads, D, page, kl, vl, min(kg, D), min(vg or kg, D), k_seed=21, v_seed=22)
        order = g.permutation(pages).astype(np.int32)
        self.table = np.full((len(lens), max(need + [1])), -7, dtype=np.int32)
        slots, at = [], 0
        for b, n in enumerate(lens):
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
            j = np.arange(n)
            slots.append(self.table[b, j // page].astype(np.int64) * page + j % page)
        self.lens, self.heads, self.D, self.page = list(lens), heads, D, page
        self.slots = slots
        flat = np.concatenate(slots) if slots else np.zeros(0, dtype=np.int64)
        k = torch.from_numpy(g.standard_normal((len(flat), heads, D)).astype(np.float32)).cuda()
        v = torch.from_numpy(g.standard_normal((len(flat), heads, D)).astype(np.float32)).cuda()
        k *= torch.from_numpy(np.exp(0.3 * g.standard_normal((len(flat), heads, 1))).astype(np.float32)).cuda()
        if vscale is not None:
            v *= torch.from_numpy(vscale(len(flat)).astype(np.float32)).cuda()[:, None, None]
        tq.kv_store(self.cache, k.to(dt), v.to(dt), torch.from_numpy(flat).cuda())
        torch.cuda.synchronize()
        self.refresh()

    def refresh(self):
        c = self.cache
        self.rows = []
        for half in (c.k, c.v):
            codes = torch_to_np(half.codes).reshape(half.E, self.heads, self.page, -1)
            scales = torch_to_np(half.scales).reshape(half.E, self.heads, self.page, -1)
            per = []
            for s in self.slots:
                cc = codes[s // self.page, :, s % self.page].reshape(len(s) * self.heads, codes.shape[-1])
                ss = scales[s // self.page, :, s % self.page].reshape(len(s) * self.heads, scales.shape[-1])
                w = oenc.dequant(cc, ss, half.levels, half.group, self.D) if len(s) else np.zeros((0, self.D))
                per.append(w.reshape(len(s), self.heads, self.D))
            self.rows.append(per)

    def dev(self):
        return (torch.tensor(self.lens, dtype=torch.int32, device="cuda"), torch.from_numpy(self.table).cuda())


def queries(M, H, D, dt, seed=0):
    g = np.random.default_rng([seed, M, H, D])
    return torch.from_numpy(g.standard_normal((M, H, D)).astype(np.float32)).cuda().to(dt)


def check(got, bt, q, counts, scale, tree=None, only=None):
    """got [M, H, D] against the oracle for the sequences' rows (counts[b] each)."""
    out = as_f64(got)
    D, H = bt.D, q.shape[1]
    share = H // bt.heads
    qr = ohd.rotate(as_f64(q).reshape(-1, D), 21).reshape(q.shape)
    m, worst = 0, 0.0
    for b, n in enumerate(counts):
        for i in range(n):
            if only is None or m in only:
                mask = oat.seen(bt.lens[b], n, i, None if tree is None else tree[m])
                for h in range(H):
                    kp, vp = bt.rows[0][b][:, h // share], bt.rows[1][b][:, h // share]
                    ref, p = oat.attend(qr[m, h], kp, vp, scale, mask)
                    want = ohd.unrotate(ref[None], 22)[0]
                    if not mask.any():
                        assert not out[m, h].any(), (m, h)
                        continue
                    kk, vv, pp = kp[mask], vp[mask], p[mask]
                    s = scale * (kk @ qr[m, h])
                    E = abs(scale) * ((3 * U + (D + 16) * 2.0 ** -24) * (np.abs(kk) @ np.abs(qr[m, h]))
                                      + 2.0 ** -19 * np.abs(qr[m, h]).max() * np.abs(kk).sum(1)) + 2.0 ** -21 * np.abs(s)
                    rel = np.expm1(2 * E.max()) + 3 * U + 2.0 ** -18 + len(s) * 2.0 ** -24
                    room = rel * np.linalg.norm(pp @ np.abs(vv)) + HALF_STEP[got.dtype] * np.linalg.norm(want) * 1.01 + 1e-7
                    err = np.linalg.norm(out[m, h] - want)
                    worst = max(worst, err / room)
                    assert err <= room, (m, h, err, room)
            m += 1
    return worst


def run(bt, q, counts=None, tree=None, **kw):
    lens, table = bt.dev()
    off = None
    if counts is not None:
        off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    words = None
    if tree is not None:
        bits = np.asarray(tree, dtype=np.uint8)
        wide = -(-bits.shape[1] // 32) * 32
        bits = np.pad(bits, ((0, 0), (0, wide - bits.shape[1])))
        words = torch.from_numpy(np.packbits(bits, axis=1, bitorder="little").view(np.int32).copy()).cuda()
    got = tq.kv_attend(bt.cache, q, lens, table, q_offsets=off, tree=words, **kw)
    torch.cuda.synchronize()
    return got


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kl,vl", [(256, 8), (16, 16), (8, 4), (4, 256), (256, 256), (16, 8)])
def test_single_tokens(D, kl, vl):
    lens = [1, 2, 15, 16, 17, 31, 33, 64, 100, 257]
    bt = Batch(lens, heads=2, D=D, page=16, kl=kl, vl=vl, seed=kl + vl)
    q = queries(len(lens), 6, D, torch.bfloat16)
    check(run(bt, q), bt, q, [1] * len(lens), D ** -0.5)


@pytest.mark.parametrize("kg,vg", [(32, 32), (32, 128), (64, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_groups(D, kg, vg):
    bt = Batch([70, 5, 200], heads=2, D=D, page=32, kg=min(kg, D), vg=min(vg, D), seed=kg)
    q = queries(3, 4, D, torch.float16)
    check(run(bt, q), bt, q, [1] * 3, D ** -0.5)


@pytest.mark.parametrize("heads,share", [(1, 1), (1, 16), (1, 17), (2, 3), (8, 8), (1, 71), (3, 32)])
def test_head_shares(heads, share):
    bt = Batch([130, 47], heads=heads, D=64, page=48, kg=32)
    q = queries(2, heads * share, 64, torch.bfloat16)
    check(run(bt, q), bt, q, [1, 1], 0.125)


@pytest.mark.parametrize("share", [1, 3, 4, 8])
@pytest.mark.parametrize("counts,lens", [([5, 1, 0, 33], [9, 300, 4, 33]), ([64, 100], [64, 401]), ([130], [131]), ([2, 2], [1, 0])])
def test_prompt_chunks_are_causal(share, counts, lens):
    bt = Batch(lens, heads=2, D=64, page=16, kg=64)
    q = queries(sum(counts), 2 * share, 64, torch.bfloat16)
    check(run(bt, q, counts), bt, q, counts, 0.125)


def test_longer_chunk_and_wide_heads():
    counts, lens = [300, 77], [1111, 500]
    for D in (128, 256):
        bt = Batch(lens, heads=1, D=D, page=64, seed=D)
        q = queries(sum(counts), 4, D, torch.bfloat16)
        only = set(range(0, 377, 23)) | {0, 299, 300, 376}
        check(run(bt, q, counts), bt, q, counts, D ** -0.5, only=only)


def test_uniform_counts_without_offsets():
    bt = Batch([40, 20, 90], heads=2, D=128, page=16)
    q = queries(12, 4, 128, torch.bfloat16)
    assert torch.equal(run(bt, q), run(bt, q, [4, 4, 4]))


def tree_rows(counts, g, words_bits):
    rows = []
    for n in counts:
        base = len(rows)
        for i in range(n):
            r = np.zeros(words_bits, dtype=np.uint8)
            if i:
                r |= rows[base + int(g.integers(0, i))]
            r[i] = 1
            rows.append(r)
    return np.stack(rows)


@pytest.mark.parametrize("D,share", [(64, 4), (128, 1), (128, 8), (256, 3)])
@pytest.mark.parametrize("counts,lens", [([7, 24, 1], [7, 600, 55]), ([60, 33], [61, 1000])])
def test_trees(D, share, counts, lens):
    bt = Batch(lens, heads=2, D=D, page=32, vl=16)
    tree = tree_rows(counts, np.random.default_rng(D), 64)
    q = queries(sum(counts), 2 * share, D, torch.float16)
    only = set(range(0, sum(counts), 5)) | {0, sum(counts) - 1}
    check(run(bt, q, counts, tree), bt, q, counts, D ** -0.5, tree, only)


def test_trees_that_leave_nothing_and_bits_past_the_words():
    # no context and an empty mask row: zeros; own tokens past the mask's words are unseen
    counts, lens = [40, 3], [40, 3]
    bt = Batch(lens, heads=1, D=64, page=16, kg=32)
    tree = np.zeros((43, 32), dtype=np.uint8)
    tree[5, 2] = 1
    tree[39, :] = 1
    tree[41, 1] = 1
    q = queries(43, 2, 64, torch.bfloat16)
    got = run(bt, q, counts, tree)
    check(got, bt, q, counts, 0.125, tree)
    assert not got[0].any() and got[5].any() and got[39].any()


def loud(bt, b, j, factor=1000.0):
    """Token j of sequence b gets values `factor` times as large (its scales)."""
    s = int(bt.slots[b][j])
    c = bt.cache.v.scales.view(-1, bt.heads, bt.page, bt.D // bt.cache.v.group)
    c[s // bt.page, :, s % bt.page] *= factor
    bt.refresh()


@pytest.mark.parametrize("j", [0, 15, 16, 31, 32, 99, 100, 101, 103])
def test_one_loud_token_is_seen_by_its_successors_alone(j):
    # the mask moved by one token anywhere near j would show a thousandfold
    bt = Batch([104], heads=1, D=64, page=16, kg=32)
    loud(bt, 0, j)
    counts = [8]
    q = queries(8, 2, 64, torch.bfloat16)
    got = run(bt, q, counts)
    check(got, bt, q, counts, 0.125)
    # an output is a mean of the values it sees: without the loud token no longer than the longest
    # of the others (1.02: the roundings); with it the bound of check() above holds the loud part
    longest = 1.02 * float(np.delete(np.linalg.norm(bt.rows[1][0][:, 0], axis=1), j).max())
    size = got.float().norm(dim=-1).amax(-1)
    for i in range(8):
        assert j <= 96 + i or float(size[i]) <= longest
    tree = np.tril(np.ones((8, 32), dtype=np.uint8))
    if j >= 96:
        tree[:, j - 96] = 0
        tree[3, j - 96] = 1
        quiet = run(bt, q, counts, tree)
        check(quiet, bt, q, counts, 0.125, tree)
        loud_rows = quiet.float().norm(dim=-1).amax(-1) > longest
        assert not any(loud_rows.tolist()[i] for i in range(8) if i != 3)


@pytest.mark.parametrize("spread", [1e-4, 1.0, 3e3])
def test_values_of_any_size(spread):
    # scales from fp16's subnormals to near its largest value, growing and shrinking along the
    # sequence: neither overflow nor lost small sequences
    n = 300
    for shape in (lambda m: np.full(m, spread), lambda m: np.geomspace(spread * 0.01, spread * 10, m),
                  lambda m: np.geomspace(spread * 10, spread * 0.01, m)):
        bt = Batch([n], heads=1, D=128, page=64, vl=256, dt=torch.float32, vscale=shape)
        q = queries(1, 3, 128, torch.bfloat16)
        lens, table = bt.dev()
        got = tq.kv_attend(bt.cache, q, lens, table)
        torch.cuda.synchronize()
        check(got, bt, q, [1], 128 ** -0.5)


@pytest.mark.parametrize("qsize", [0.0, 1e-6, 30.0, 300.0])
def test_queries_of_any_size(qsize):
    bt = Batch([500, 3], heads=2, D=64, page=16, kg=32)
    q = queries(2, 4, 64, torch.bfloat16) * qsize
    check(run(bt, q), bt, q, [1, 1], 0.125)


def test_negative_and_zero_scale():
    bt = Batch([90], heads=1, D=64, page=16, kg=32)
    q = queries(1, 2, 64, torch.bfloat16)
    for s in (0.0, -0.2):
        check(run(bt, q, scale=s), bt, q, [1], s)


def test_bad_pages_poison_their_readers_alone():
    bt = Batch([100, 100], heads=2, D=64, page=16, kg=32)
    q = queries(6, 4, 64, torch.bfloat16)
    want = run(bt, q, [3, 3])
    for bad in (-1, bt.cache.k.E, 2 ** 31 - 1, -2 ** 31):
        table = bt.table.copy()
        bt.table[0, 6] = bad                # tokens 96 .. 99 of sequence 0
        got = run(bt, q, [3, 3])
        bt.table[:] = table
        assert torch.isnan(got[:3]).all()
        assert torch.equal(got[3:], want[3:])
    # queries that stop before the bad page do not see it
    bt.lens[0] = 96
    table = bt.table.copy()
    bt.table[0, 6] = -1
    got = run(bt, q, [3, 3])
    bt.table[:] = table
    assert not torch.isnan(got).any()


def test_nan_and_infinite_rows_reach_their_readers_alone():
    bt = Batch([64, 64], heads=1, D=64, page=16, kg=32)
    q = queries(4, 2, 64, torch.bfloat16)
    want = run(bt, q, [2, 2])
    for part in (bt.cache.k, bt.cache.v):
        keep = part.scales.clone()
        s = int(bt.slots[0][63])
        part.scales.view(-1, 1, 16, 2)[s // 16, :, s % 16] = float("nan")
        got = run(bt, q, [2, 2])
        assert torch.equal(got[0], want[0]) and torch.equal(got[2:], want[2:])   # query 0 stops at token 62
        assert torch.isnan(got[1]).all()
        part.scales.copy_(keep)
    # unused rows of the last page may hold anything
    for part in (bt.cache.k, bt.cache.v):
        keep = part.scales.clone()
        part.scales.fill_(float("nan"))
        for b in range(2):
            for s in bt.slots[b]:
                part.scales.view(-1, 1, 16, 2)[s // 16, :, s % 16] = keep.view(-1, 1, 16, 2)[s // 16, :, s % 16]
    assert torch.equal(run(bt, q, [2, 2]), want)


def test_lengths_outside_the_table_are_cut():
    bt = Batch([48, 20], heads=1, D=64, page=16, kg=32)
    q = queries(2, 2, 64, torch.bfloat16)
    want = run(bt, q)
    bt.lens = [1000, 20]        # table of 3 pages: 48 tokens
    assert torch.equal(run(bt, q), want)
    bt.lens = [48, -5]
    got = run(bt, q)
    assert torch.equal(got[0], want[0]) and not got[1].any()


def test_rows_behind_the_last_sequence_stay():
    bt = Batch([30, 40], heads=1, D=64, page=16, kg=32)
    q = queries(9, 2, 64, torch.bfloat16)
    out = torch.full((9, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lens, table = bt.dev()
    off = torch.tensor([0, 2, 5], dtype=torch.int32, device="cuda")
    tq.kv_attend(bt.cache, q, lens, table, q_offsets=off, out=out)
    torch.cuda.synchronize()
    check(out[:5], bt, q[:5], [2, 3], 0.125)
    assert torch.all(out[5:] == 7.0)


def test_strided_queries_and_output_types():
    bt = Batch([50, 60], heads=2, D=128, page=16)
    wide = queries(2, 12, 128, torch.bfloat16)
    q = wide[:, :4]             # a slice of a fused projection
    want = run(bt, q.contiguous())
    assert torch.equal(run(bt, q), want)
    half = run(bt, q, out_dtype=torch.float16)
    check(half, bt, q, [1, 1], 128 ** -0.5)


@pytest.mark.parametrize("B", [1, 3, 300])
def test_many_and_few_sequences(B):
    g = np.random.default_rng(B)
    lens = [int(x) for x in g.integers(0, 90, B)]
    bt = Batch(lens, heads=1, D=64, page=16, kg=32)
    q = queries(B, 2, 64, torch.bfloat16)
    check(run(bt, q), bt, q, [1] * B, 0.125)


def test_a_long_sequence():
    bt = Batch([40000, 17, 9000], heads=2, D=128, page=256)
    q = queries(3, 8, 128, torch.bfloat16)
    check(run(bt, q), bt, q, [1] * 3, 128 ** -0.5)


def test_calls_repeat_bit_for_bit():
    bt = Batch([3000, 17, 900], heads=2, D=128, page=64)
    q = queries(30, 8, 128, torch.bfloat16)
    first = run(bt, q, [10, 10, 10])
    for _ in range(3):
        assert torch.equal(run(bt, q, [10, 10, 10]), first)


def test_two_streams_with_their_own_workspaces():
    bt = Batch([5000, 17], heads=2, D=128, page=64)
    qs = [queries(2, 8, 128, torch.bfloat16, seed=s) for s in range(2)]
    want = [run(bt, q) for q in qs]
    lens, table = bt.dev()
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in qs], [[], []]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(tq.kv_attend(bt.cache, qs[i], lens, table))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])


def test_a_decode_step_captured_and_replayed():
    # rope on the queries, store with rope on the keys, attend: one captured step, replayed with
    # new tokens, against the same calls made eagerly
    heads, H, D, page, B = 2, 8, 128, 16, 3
    bt = Batch([50, 33, 16], heads=heads, D=D, page=page, spare=6)
    r = tq.rope_frequencies(D)
    table = np.concatenate([bt.table, np.full((B, 1), -1, dtype=np.int32)], axis=1)
    free = [p for p in range(bt.cache.k.E) if p not in set(table.reshape(-1).tolist())]
    for b in range(B):
        table[b, -(-bt.lens[b] // page)] = free[b]
    table = torch.from_numpy(table).cuda()
    lens = torch.tensor(bt.lens, dtype=torch.int32, device="cuda")
    x = torch.zeros((B, H + 2 * heads, D), dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(B, dtype=torch.int32, device="cuda")
    slots = torch.zeros(B, dtype=torch.int64, device="cuda")
    start = [t.clone() for t in (bt.cache.k.codes, bt.cache.k.scales, bt.cache.v.codes, bt.cache.v.scales)]

    def fill(rep):
        g = np.random.default_rng(rep)
        x.copy_(torch.from_numpy(g.standard_normal(tuple(x.shape)).astype(np.float32)))
        p = (lens - 1).to(torch.int64)
        pos.copy_(p)
        slots.copy_(torch.gather(table, 1, (p // page)[:, None]).squeeze(1) * page + p % page)

    def step():
        q = tq.rope(x[:, :H], pos, r)
        tq.kv_store(bt.cache, x[:, H:H + heads], x[:, H + heads:], slots, rope=r, positions=pos)
        return tq.kv_attend(bt.cache, q, lens, table)

    fill(0)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for t, s in zip((bt.cache.k.codes, bt.cache.k.scales, bt.cache.v.codes, bt.cache.v.scales), start):
        t.copy_(s)
    lens.copy_(torch.tensor(bt.lens, dtype=torch.int32))
    for rep in range(1, 5):
        lens += 1
        fill(rep)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        eager = step()       # the same tokens into the same slots: the cache is what it was
        torch.cuda.synchronize()
        assert torch.isfinite(eager).all() and torch.equal(got, eager), rep


def test_two_captured_calls_share_a_workspace_in_order():
    bt = Batch([3000, 100], heads=2, D=128, page=64)
    qs = [queries(2, 8, 128, torch.bfloat16, seed=s) for s in range(2)]
    want = [run(bt, q) for q in qs]
    lens, table = bt.dev()
    ws = torch.empty(max(1, tq.kv_attend_workspace(bt.cache, 8, 2, 2)), dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(q) for q in qs]
    graphs = []
    for q, o in zip(qs, outs):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            tq.kv_attend(bt.cache, q, lens, table, out=o, ws=ws)
        graphs.append(gr)
    for _ in range(4):
        ws.fill_(255)
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
            o.zero_()


def test_whole_path_against_plain_attention():
    # rope, store, attend over a prompt and then single tokens, against attention of the
    # unquantized keys and values: 8-bit keys and values keep the outputs within the codebook's
    # distortion (relative squared error 4.1e-5 each; the keys' enters through the scores)
    g = np.random.default_rng(77)
    heads, H, D, page, n = 2, 4, 64, 16, 70
    c = tq.kv_cache(6, heads, D, page, 256, 256, 64, 64, k_seed=1, v_seed=2)
    r = tq.rope_frequencies(D)
    x = torch.from_numpy(g.standard_normal((n, H + 2 * heads, D)).astype(np.float32)).cuda().to(torch.bfloat16)
    pos = torch.arange(n, device="cuda")
    table = torch.from_numpy(g.permutation(6).astype(np.int32)[None]).cuda()
    slots = table[0, (pos // page)].to(torch.int64) * page + pos % page
    qt = tq.rope(x[:, :H], pos, r)
    f = as_f64(x)
    k = oat.rope(f[:, H:H + heads], np.arange(n), r.inv_freq.cpu().numpy(), D)
    outs = []
    for a, b in ((0, 64), (64, 65), (65, 66), (66, 70)):
        tq.kv_store(c, x[a:b, H:H + heads], x[a:b, H + heads:], slots[a:b], rope=r, positions=pos[a:b])
        outs.append(tq.kv_attend(c, qt[a:b], torch.tensor([b], dtype=torch.int32, device="cuda"), table))
    torch.cuda.synchronize()
    got, q = as_f64(torch.cat(outs)), as_f64(qt)
    want = np.zeros_like(got)
    for i in range(n):
        for h in range(H):
            want[i, h], _ = oat.attend(q[i, h], k[:, h // 2], f[:, H + heads + h // 2], D ** -0.5, np.arange(n) <= i)
    err = np.sum((got - want) ** 2) / np.sum(want ** 2)
    # both distortions, scores of unit size (factor up to 2 on the keys' part), bf16 roundings 2^-16 / 3 each
    assert err < 4.1e-5 * 3 + 2 * 2.0 ** -16, err
