"""Attention over the packed cache where the scales of neighbouring rows differ by what fp16 cannot
hold at once, and where rows that nobody may read hold anything. The bounds are those of
test_gpu_kv_attend.
"""

import numpy as np
import pytest
import torch

import rotation_lloyd_max_amd as tq
from oracle import attention as oat
from oracle import hadamard as ohd
from parity import as_f64
from test_gpu_kv_attend import HALF_STEP, U, Batch, check, queries, run

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


def check_rows(out, bt, q, counts, scale, seq, rows, tree=None):
    """Rows of sequence `seq` against the oracle, by the bound of test_gpu_kv_attend's docstring with two
    changes. Only the tokens that can have weight enter its largest score error E: one whose score, errors
    E_j included, lies 60 below the largest has weight e^-60 at most, whatever the others'. And the
    weights' own floor is counted: fp16's subnormals cut 2^-25 of a weight held against 2^7, so 2^-32 of
    each value with weight above e^-60. Nothing else is allowed: outputs in bf16, whose range holds any."""
    got, D, H = as_f64(out), bt.D, q.shape[1]
    share, m0 = H // bt.heads, sum(counts[:seq])
    for i in rows:
        m, mask = m0 + i, oat.seen(bt.lens[seq], counts[seq], i, None if tree is None else tree[m0 + i])
        qr = ohd.rotate(as_f64(q[m]), 21)
        for h in range(H):
            kp, vp = bt.rows[0][seq][mask, h // share], bt.rows[1][seq][mask, h // share]
            ref, p = oat.attend(qr[h], kp, vp, scale, np.ones(len(kp), dtype=bool))
            want = ohd.unrotate(ref[None], 22)[0]
            s = scale * (kp @ qr[h])
            E = abs(scale) * ((3 * U + (D + 16) * 2.0 ** -24) * (np.abs(kp) @ np.abs(qr[h]))
                              + 2.0 ** -19 * np.abs(qr[h]).max() * np.abs(kp).sum(1)) + 2.0 ** -21 * np.abs(s)
            best = np.argmax(s)
            heavy = s + E > s[best] - E[best] - 60
            rel = np.expm1(2 * E[heavy].max()) + 3 * U + 2.0 ** -18 + len(s) * 2.0 ** -24
            room = rel * np.linalg.norm(p @ np.abs(vp)) + 2.0 ** -32 * np.linalg.norm(np.abs(vp[heavy]).sum(0))
            room += HALF_STEP[out.dtype] * np.linalg.norm(want) * 1.01
            err = np.linalg.norm(got[m, h] - want)
            assert err <= room, (m, h, err, room)


LONG = 600      # tokens of the first sequence
ROWS = [(5, 3), (40, 2), (150, 2)]      # queries of a sequence, query heads per key head: as TILES


def mixed(D, n, share, low, high, seed):
    """A long sequence among short ones (so many for tiles of 16 that each wave takes several blocks of the
    long one in turn), all scales spread from low to high."""
    lens = [LONG] + [n] * (140 if n == ROWS[0][0] else 2)
    bt = Batch(lens, heads=1, D=D, page=48, kg=32, vg=64, kl=256, vl=256, seed=seed, dt=torch.float32)
    g = torch.Generator(device="cuda").manual_seed(seed)
    for part in (bt.cache.k, bt.cache.v):
        u = torch.empty(part.scales.shape, device="cuda").uniform_(np.log(low), np.log(high), generator=g)
        part.scales.copy_(torch.exp(u))
    return bt, [n] * len(lens), queries(n * len(lens), share, D, torch.bfloat16, seed=seed)


def make_loud(bt, tokens, scale, same_key):
    """The scales of some tokens of sequence 0; same_key: with the codes of the first one's key."""
    for j in tokens:
        s, first = int(bt.slots[0][j]), int(bt.slots[0][tokens[0]])
        for part in (bt.cache.k, bt.cache.v):
            scales_of(bt, part)[s // bt.page, :, s % bt.page] = scale
        if same_key:
            c = bt.cache.k.codes.view(-1, bt.heads, bt.page, bt.cache.k.codes.shape[-1])
            c[s // bt.page, :, s % bt.page] = c[first // bt.page, :, first % bt.page].clone()
    bt.refresh()


# Scales of the others from, to, and the size of the queries: small ones, so that all weights are nearly
# equal and the values' errors show, and ones that bring the scores to a few units, so that the keys' do.
# Beside a scale of 3e4 all of these would be held in fp16 by few bits or none.
LOUD = 3e4
SPREADS = [(2e-4, 5e-4, 0.01), (3e-7, 2e-5, 0.3), (1e-3, 3e-3, 3e3)]


@pytest.mark.parametrize("low,high,size", SPREADS)
@pytest.mark.parametrize("n,share", ROWS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_loud_tokens_hidden_by_a_tree_cost_the_others_nothing(D, n, share, low, high, size):
    bt, counts, q = mixed(D, n, share, low, high, D + n)
    q = q * size
    own = [n - 3] if n < 40 else [2, n // 2, n - 3]        # the sequence's own tokens, by its mask's bits
    make_loud(bt, [LONG - n + i for i in own], LOUD, False)
    tree = np.tile(np.tril(np.ones((n, n), dtype=np.uint8)), (len(counts), 1))
    tree[:n, own] = 0
    tree[1, own] = 1
    out = run(bt, q, counts, tree)
    rows = [0, 2, n - 1] if n < 40 else [0, 2, 3, n // 2 - 1, n // 2, n // 2 + 1, n - 4, n - 1]
    check_rows(out, bt, q, counts, D ** -0.5, 0, rows, tree)


@pytest.mark.parametrize("low,high,size", SPREADS)
@pytest.mark.parametrize("at", [[3], [70, 71, 200, 333], [LONG - 2]])
@pytest.mark.parametrize("n,share", ROWS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_loud_tokens_without_weight_cost_the_others_nothing(D, n, share, at, low, high, size):
    # every query is turned away from the loud tokens' key: they are seen, with weights that fp32 has as 0
    bt, counts, q = mixed(D, n, share, low, high, D + n + len(at))
    make_loud(bt, at, LOUD, True)
    away = ohd.unrotate(bt.rows[0][0][at[0]], 21)[0]
    away = torch.from_numpy(away / np.linalg.norm(away) * D ** 0.5).to(q)
    q = (q - away) * size
    out = run(bt, q, counts)
    check_rows(out, bt, q, counts, D ** -0.5, 0, sorted({0, 1, n // 2, n - 2, n - 1}))
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("n,share", ROWS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_values_of_every_size_side_by_side(D, n, share):
    # value scales over all of fp16's range in every block, weights near each other
    bt, counts, q = mixed(D, n, share, 1e-7, 5e4, D + n)
    bt.cache.k.scales.fill_(0.5)
    bt.refresh()
    out = run(bt, q, counts)
    check_rows(out, bt, q, counts, D ** -0.5, 0, [0, n // 2, n - 1])


@pytest.mark.parametrize("n,share", ROWS)
def test_a_value_that_is_no_number_beside_loud_and_quiet_ones(n, share):
    bt, counts, q = mixed(128, n, share, 1e-7, 5e4, n)
    bt.cache.k.scales.fill_(0.5)
    bt.refresh()
    want = run(bt, q, counts)
    for bits in (0x7e00, 0x7c00):
        keep = bt.cache.v.scales.clone()
        s = int(bt.slots[0][LONG - 2])
        scales_of(bt, bt.cache.v).view(torch.int16)[s // bt.page, :, s % bt.page] = bits
        got = run(bt, q, counts)
        bt.cache.v.scales.copy_(keep)
        same = torch.equal(got[:n - 2], want[:n - 2]) and torch.equal(got[n:], want[n:])
        assert same and torch.isnan(got[n - 2:n]).all(), bits


@pytest.mark.parametrize("n,share", ROWS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_of_zeros(D, n, share):
    # a scale of 0 (a key or value of zeros) alone, beside others, and in a whole cache
    bt, counts, q = mixed(D, n, share, 0.1, 2.0, D + n)
    for part, step in ((bt.cache.k, 5), (bt.cache.v, 7)):
        for j in range(0, LONG, step):
            s = int(bt.slots[0][j])
            scales_of(bt, part)[s // bt.page, :, s % bt.page] = 0.0
    bt.refresh()
    check_rows(run(bt, q, counts), bt, q, counts, D ** -0.5, 0, [0, n // 2, n - 1])
    bt.cache.k.scales.zero_()
    bt.refresh()
    check_rows(run(bt, q, counts), bt, q, counts, D ** -0.5, 0, [0, n - 1])
    bt.cache.v.scales.zero_()
    assert not run(bt, q, counts).any()


@pytest.mark.parametrize("n,share", ROWS)
def test_captured_calls_with_scales_of_every_size(n, share):
    bt, counts, q = mixed(128, n, share, 1e-7, 5e4, n)
    bt.cache.k.scales.fill_(0.5)
    lens, table = bt.dev()
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    tq.kv_attend(bt.cache, q, lens, table, q_offsets=off)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = tq.kv_attend(bt.cache, q, lens, table, q_offsets=off)
    for rep in range(4):
        bt.cache.v.scales.mul_(0.25 if rep % 2 else 0.5)
        q.copy_(queries(*q.shape, torch.bfloat16, seed=rep))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        same = torch.equal(out, tq.kv_attend(bt.cache, q, lens, table, q_offsets=off))
        assert same and torch.isfinite(out).all(), rep
