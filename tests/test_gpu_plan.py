"""A step's tables and what stays of it (tq_kv_plan, tq_kv_keep) on the GPU against the oracle: whole
numbers, equal throughout."""

import numpy as np
import pytest
import torch

import rotation_lloyd_max_amd as tq
from oracle import step as ost

pytestmark = pytest.mark.gpu


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(x)).to(dtype).cuda()


def setup(g, lens, page, pages, width, free=None):
    """A table that holds lens, and the list of the other pages (free of them on it)."""
    order = [int(x) for x in g.permutation(pages)]
    table = np.full((len(lens), width), -1)
    for b, n in enumerate(lens):
        for j in range(-(-max(0, int(n)) // page)):
            if j < width:
                table[b, j] = order.pop()
    return table, order if free is None else order[:free]


def pool_of(free, pages):
    stack = torch.full((pages,), -5, dtype=torch.int32)
    stack[:len(free)] = torch.tensor(free, dtype=torch.int32)
    return tq.KVPool(stack.cuda(), torch.tensor([len(free), 0], dtype=torch.int32, device="cuda"))


def check_plan(lens, counts, table, free, rows, page, pages, parents=None, words=0, shift=None, look=False):
    want = ost.plan(free, lens, counts, table, rows, page, pages, parents, words, shift)
    pool, t = pool_of(free, pages), dev(table)
    left = torch.full((1,), 77, dtype=torch.int32, device="cuda") if look else None
    p = tq.kv_plan(pool, dev(lens), dev(counts), t, rows, page, parents=None if parents is None else dev(parents),
                   tree_words=words, shift=None if shift is None else dev(shift), left=left)
    torch.cuda.synchronize()
    for name in ("slots", "positions", "q_offsets", "kv_lens", "status"):
        got = getattr(p, name).cpu().numpy()
        assert np.array_equal(got, want[name]), (name, got, want[name])
    if words:
        assert np.array_equal(p.tree.cpu().numpy().view(np.uint32), want["tree"])
    else:
        assert p.tree is None
    assert np.array_equal(t.cpu().numpy(), want["table"])
    assert pool.state.tolist() == [len(free) if look else len(want["free"]), 0]
    assert not look or left.item() == len(want["free"])
    assert pool.free[:len(free)].tolist() == list(free)
    return want, pool, t, p


def chains(counts):
    return np.concatenate([np.arange(-1, max(0, c) - 1) for c in counts] or [np.zeros(0)]).clip(min=0).astype(np.int64)


def trees(g, counts, reach=4):
    return np.concatenate([[0] + [int(g.integers(max(0, i - reach), i)) for i in range(1, c)] if c > 0 else [] for c in counts]
                          or [np.zeros(0)]).astype(np.int64)


@pytest.mark.parametrize("B,longest,most,page", [
    (1, 0, 1, 64), (1, 100, 1, 16), (3, 70, 5, 16), (16, 4000, 1, 64), (64, 300, 9, 32), (65, 1000, 33, 16), (5, 3000, 4001, 32),
    (1023, 40, 3, 16), (1024, 40, 3, 16), (1025, 90, 3, 16), (3000, 30, 4, 16), (2, 5000, 9000, 256), (7, 100, 40, 1), (300, 9, 9, 3)])
@pytest.mark.parametrize("tree", [False, True])
def test_plan_matches_oracle(B, longest, most, page, tree):
    g = np.random.default_rng([B, longest, most, page])
    lens, counts = g.integers(0, longest + 1, B), g.integers(0, most + 1, B)
    width = -(-(longest + most) // page)
    pages = int(sum(-(-lens // page))) + int(sum(-(-(lens + counts) // page))) + 3
    table, free = setup(g, lens, page, pages, width)
    rows = int(counts.sum()) + 3
    shift = g.integers(-99, 99, B)
    if tree and counts.sum():
        p = np.concatenate([trees(g, counts), [0, 0, 0]])
        check_plan(lens, counts, table, free, rows, page, pages, p, (max(counts) + 31) // 32, shift)
    else:
        check_plan(lens, counts, table, free, rows, page, pages, shift=shift)
        check_plan(lens, counts, table, free, rows, page, pages, words=2, look=True)


@pytest.mark.parametrize("seed", range(6))
def test_sequences_that_are_refused(seed):
    # too few pages, rows or table entries, negative lengths and counts, pages that are none
    g = np.random.default_rng(100 + seed)
    B, page = 40, 16
    lens, counts = g.integers(-20, 200, B), g.integers(-3, 40, B)
    width = 11
    table, free = setup(g, np.minimum(lens, width * page), page, 700, width, free=[0, 1, 5, 20, 33, 700][seed])
    if len(free) > 3:
        free[2], free[-1] = -1, 4000
    held = np.nonzero(table >= 0)
    table[held[0][::7], held[1][::7]] = [-1, 700, 2 ** 30][seed % 3]
    total = int(np.maximum(counts, 0).sum())
    for rows in (0, 1, total // 2, total, total + 100):
        check_plan(lens, counts, table, free, rows, page, 700, look=seed % 2 == 0)
        check_plan(lens, counts, table, free, rows, page, 700, np.zeros(rows, int), 1)
    w = ost.plan(free, lens, counts, table, total // 2, page, 700)
    assert len(set(w["status"])) >= 3 or seed > 3


def test_parents_that_are_none_end_the_walk():
    parents = np.array([5, 0, 1, 3, 9, -1, 2, 6, 1 << 20])
    check_plan([20], [9], np.array([[3, 1, -1]]), [0, 2], 9, 16, 4, parents, 1)
    check_plan([20], [9], np.array([[3, 1, -1]]), [0, 2], 9, 16, 4, parents, 2)


@pytest.mark.parametrize("n,words", [(70, 2), (70, 3), (2100, 66), (2100, 5), (4500, 141)])
def test_long_trees_and_masks_cut_short(n, words):
    # (more parents than the workgroups hold, ancestors in words that are left out)
    g = np.random.default_rng(n)
    counts = [3, n, 5]
    lens = [7, 100, 0]
    table, free = setup(g, lens, 64, 200, 90)
    for p in (trees(g, counts), trees(g, counts, reach=n), chains(counts)):
        check_plan(lens, counts, table, free, sum(counts), 64, 200, p, words)


def test_no_sequences_and_no_rows():
    check_plan([], [], np.zeros((0, 4), int), [1, 2], 5, 16, 9)
    check_plan([], [], np.zeros((0, 0), int), [], 0, 16, 9)
    check_plan([3, 0], [0, 0], np.array([[1], [2]]), [4], 0, 16, 9)


def test_longest_sequences():
    # lengths near the largest: a table row of 2^31 - 65536 - 16 tokens in pages of 65536
    width, page = 32766, 65536
    table = np.full((2, width), -1)
    table[0, :32765] = np.arange(32765)
    lens = [32765 * page, 5]
    table[1, 0] = 40000
    check_plan(lens, [page, 3], table, [50001, 50000], page + 3, page, 60000)
    check_plan([32766 * page, 2 ** 31 - 1], [1, 2 ** 31 - 1], table, [50001], 10, page, 60000)


# ---- what stays ---------------------------------------------------------------------------

def filled(pages, heads, D, page, kl, vl, group, seed):
    c = tq.kv_cache(pages, heads, D, page_tokens=page, k_levels=kl, v_levels=vl, k_group=group, v_group=group)
    g = torch.Generator(device="cuda").manual_seed(seed)
    for w in (c.k, c.v):
        w.codes.copy_(torch.randint(-2 ** 31, 2 ** 31 - 1, w.codes.shape, generator=g, device="cuda", dtype=torch.int32))
        w.scales.copy_(torch.rand(w.scales.shape, generator=g, device="cuda").to(torch.float16))
    return c


def moved(cache, page, heads, table, lens, q_offsets, path, moves):
    """The four tensors after the moves, one row after another."""
    out = [t.clone() for w in (cache.k, cache.v) for t in (w.codes, w.scales)]
    pages = cache.k.E
    for b, j in moves:
        src = int(path[q_offsets[b] + j])
        if not j < src < q_offsets[b + 1] - q_offsets[b]:
            continue
        s, d = lens[b] + src, lens[b] + j
        sp, dp = table[b][s // page], table[b][d // page]
        if 0 <= sp < pages and 0 <= dp < pages:
            for t in out:
                t[dp, d % page::page] = t[sp, s % page::page].clone()
    return out


def branch(g, n):
    """An ascending path from the root, dense enough that places are sources of later rows too."""
    k = int(g.integers(1, n + 1))
    return [0] + sorted(int(x) for x in g.choice(np.arange(1, n), k - 1, replace=False))


@pytest.mark.parametrize("B,most,heads,D,kl,vl,group,page", [
    (1, 2, 1, 64, 256, 4, 32, 16), (3, 9, 2, 64, 8, 8, 32, 16), (16, 24, 8, 128, 256, 8, 64, 64), (5, 60, 3, 256, 16, 256, 128, 16),
    (40, 7, 5, 128, 4, 16, 64, 32), (2, 200, 1, 64, 256, 256, 64, 16), (9, 12, 37, 128, 256, 8, 32, 16)])
@pytest.mark.parametrize("in_place", [False, True])
def test_keep_matches_oracle(B, most, heads, D, kl, vl, group, page, in_place):
    g = np.random.default_rng([B, most, heads, D])
    lens, counts = g.integers(0, 200, B), g.integers(1, most + 1, B)
    width = -(-(200 + most) // page)
    pages = int(sum(-(-(lens + counts) // page))) + 4
    table, free = setup(g, lens, page, pages, width)
    want, pool, t, p = check_plan(lens, counts, table, free, int(counts.sum()), page, pages)
    cache = filled(pages, heads, D, page, kl, vl, group, B)
    paths = [branch(g, int(c)) for c in counts]
    kept = np.array([len(x) for x in paths])
    kept[g.random(B) < 0.2] = 0
    kept[g.random(B) < 0.2] = -1
    path = np.full(int(counts.sum()), -1)
    for b, x in enumerate(paths):
        path[want["q_offsets"][b]:want["q_offsets"][b] + len(x)] = x
    ends, stack, moves = ost.keep(want["free"], lens, kept, want["table"], page, want["q_offsets"], want["status"])
    data = moved(cache, page, heads, want["table"], lens, want["q_offsets"], path, moves)
    L = dev(lens)
    left = None if in_place else torch.zeros(1, dtype=torch.int32, device="cuda")
    out = tq.kv_keep(pool, L, dev(kept), t, page, q_offsets=p.q_offsets, status=p.status, path=dev(path), cache=cache,
                     out=L if in_place else None, left=left)
    torch.cuda.synchronize()
    assert np.array_equal(out.cpu().numpy(), ends)
    assert in_place == (out.data_ptr() == L.data_ptr()) and (in_place or np.array_equal(L.cpu().numpy(), lens))
    assert pool.state.tolist() == [len(stack) if in_place else len(want["free"]), 0]
    assert in_place or left.item() == len(stack)
    assert pool.free[:len(stack)].tolist() == stack
    for a, b in zip((cache.k.codes, cache.k.scales, cache.v.codes, cache.v.scales), data):
        assert torch.equal(a, b)


@pytest.mark.parametrize("B", [1, 1000, 1024, 1025, 2500])
def test_keep_lengths_and_pages_only(B):
    g = np.random.default_rng(B)
    page = 16
    lens, counts = g.integers(0, 300, B), g.integers(0, 40, B)
    width = 22
    pages = int(sum(-(-lens // page))) + B
    table, free = setup(g, lens, page, pages, width)
    want, pool, t, p = check_plan(lens, counts, table, free, int(counts.sum()), page, pages)
    assert B < 1000 or 1 in want["status"]
    kept = g.integers(-1, 45, B)
    ends, stack, _ = ost.keep(want["free"], lens, kept, want["table"], page, want["q_offsets"], want["status"])
    L = dev(lens)
    tq.kv_keep(pool, L, dev(kept), t, page, q_offsets=p.q_offsets, status=p.status, out=L)
    torch.cuda.synchronize()
    assert np.array_equal(L.cpu().numpy(), ends)
    assert pool.state.tolist() == [len(stack), 0] and pool.free[:len(stack)].tolist() == stack
    # the sequences end, without a plan: every page comes back, once
    tq.kv_keep(pool, L, dev(np.full(B, -1)), t, page, out=L)
    torch.cuda.synchronize()
    assert not L.any() and pool.state.tolist() == [pages, 0]
    assert sorted(pool.free.tolist()) == list(range(pages))


def test_keeping_nothing_restores_the_list():
    g = np.random.default_rng(1)
    lens, counts = g.integers(0, 100, 20), g.integers(0, 60, 20)
    table, free = setup(g, lens, 16, 400, 10)
    want, pool, t, p = check_plan(lens, counts, table, free, int(counts.sum()), 16, 400)
    pool.free[pool.state[0].item():] = -7
    out = tq.kv_keep(pool, dev(lens), dev(np.zeros(20)), t, 16, q_offsets=p.q_offsets)
    torch.cuda.synchronize()
    assert pool.state.tolist() == [len(free), 0] and pool.free[:len(free)].tolist() == free
    assert np.array_equal(out.cpu().numpy(), lens)


def test_bad_paths_and_pages_move_nothing_outside():
    # entries that do not ascend past their place, past the rows, pages that are none: those rows stay
    page, heads = 16, 2
    cache = filled(4, heads, 64, page, 256, 8, 32, 3)
    table = np.array([[1, 9, 2], [3, -1, 0]])
    lens, counts = np.array([10, 20]), np.array([12, 12])
    offsets = np.array([0, 12, 24])
    path = np.array([0, 5, 2, 4, 40, -3, 11, 7, -1, -1, -1, -1] + [0, 1, 2, 5, 3, 13, 2 ** 30, 7, 8, 9, 10, 11])
    kept = np.array([7, 9])
    moves = [(0, j) for j in range(1, 7)] + [(1, j) for j in range(1, 9)]
    data = moved(cache, page, heads, table, lens, offsets, path, moves)
    pool = pool_of([], 4)
    out = tq.kv_keep(pool, dev(lens), dev(kept), dev(table), page, q_offsets=dev(offsets), path=dev(path), cache=cache)
    torch.cuda.synchronize()
    assert out.tolist() == [17, 29]
    for a, b in zip((cache.k.codes, cache.k.scales, cache.v.codes, cache.v.scales), data):
        assert torch.equal(a, b)
    assert pool.state.tolist() == [0, 0]


def test_more_pages_than_the_pool_has_room_for():
    # (a list that was full already: nothing is written behind it)
    stack = torch.arange(6, dtype=torch.int32, device="cuda")
    pool = tq.KVPool(stack[:4], torch.tensor([3, 0], dtype=torch.int32, device="cuda"))
    out = tq.kv_keep(pool, dev([40]), dev([-1]), dev([[2, 1, 3]]), 16)
    torch.cuda.synchronize()
    assert out.item() == 0 and pool.state.tolist() == [4, 0] and stack[4:].tolist() == [4, 5]


def test_other_stream_and_int64_arguments():
    lens, counts = torch.tensor([20, 3], device="cuda"), torch.tensor([2, 5], device="cuda")
    table = torch.tensor([[4, 5, -1], [6, -1, -1]], dtype=torch.int32, device="cuda")
    pool = tq.kv_pool(4)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        p = tq.kv_plan(pool, lens, counts, table, 7, 16)
    st.synchronize()
    assert p.positions.tolist() == [20, 21, 3, 4, 5, 6, 7] and p.slots.tolist()[2:4] == [-1, -1]
    assert pool.state.tolist() == [4, 0]


def test_rows_that_the_path_does_not_have_do_not_stay():
    page, heads = 16, 2
    cache = filled(4, heads, 64, page, 256, 8, 32, 5)
    table = np.array([[1, 2], [3, 0]])
    lens, kept, path = np.array([4, 6]), np.array([3, 9]), np.array([0, 3, 5, 6, 7, 8, 9, 10, 11, 1, 1, 1, 0, 3, 7])
    want = moved(cache, page, heads, table, lens, np.array([0, 12, 15]), path, [(0, 1), (0, 2)])
    for offsets in ([0, 12, 24], [-5, 12, 2 ** 31 - 1]):
        mine = filled(4, heads, 64, page, 256, 8, 32, 5)
        out = tq.kv_keep(pool_of([], 4), dev(lens), dev(kept), dev(table), page, q_offsets=dev(offsets), path=dev(path), cache=mine)
        torch.cuda.synchronize()
        assert out.tolist() == [7, 9]
        for a, b in zip((mine.k.codes, mine.k.scales, mine.v.codes, mine.v.scales), want):
            assert torch.equal(a, b)


def test_moves_in_a_cache_of_gigabytes():
    page, heads, pages = 64, 8, 70000      # (4.6 GB of key codes)
    cache = tq.kv_cache(pages, heads, 128, page_tokens=page)
    table = np.array([[69998, 69999, 3], [1, 40000, 69997]])
    lens, path, kept = np.array([60, 126]), np.array([0, 2, 5, 6, -1, -1, -1] + [0, 1, 3, 5, 6, -1, -1]), np.array([4, 5])
    g = torch.Generator(device="cuda").manual_seed(7)
    for w in (cache.k, cache.v):
        for t in (w.codes, w.scales):
            rows = t[table.reshape(-1)]
            t[table.reshape(-1)] = torch.randint(1, 2 ** 14, rows.shape, generator=g, device="cuda").to(t.dtype)
    before = [{p: t[p].clone() for p in table.reshape(-1)} for w in (cache.k, cache.v) for t in (w.codes, w.scales)]
    for b in range(2):
        for j in range(1, kept[b]):
            s, d = lens[b] + path[7 * b + j], lens[b] + j
            for t in before:
                t[table[b][d // page]][d % page::page] = t[table[b][s // page]][s % page::page].clone()
    out = tq.kv_keep(pool_of([], pages), dev(lens), dev(kept), dev(table), page, q_offsets=dev([0, 7, 14]), path=dev(path), cache=cache)
    torch.cuda.synchronize()
    assert out.tolist() == [64, 131]
    for t, want in zip((t for w in (cache.k, cache.v) for t in (w.codes, w.scales)), before):
        assert all(torch.equal(t[p], x) for p, x in want.items())


def test_as_many_sequences_as_there_may_be():
    g = np.random.default_rng(11)
    lens, counts = g.integers(0, 50, 65536), g.integers(0, 3, 65536)
    table, free = setup(g, lens, 16, 300000, 5)
    want, pool, t, p = check_plan(lens, counts, table, free, int(counts.sum()) + 5, 16, 300000)
    kept = g.integers(-1, 4, 65536)
    ends, left, _ = ost.keep(want["free"], lens, kept, want["table"], 16, q_offsets=want["q_offsets"], status=want["status"])
    out = tq.kv_keep(pool, dev(lens), dev(kept), t, 16, q_offsets=p.q_offsets, status=p.status)
    torch.cuda.synchronize()
    assert np.array_equal(out.cpu().numpy(), ends)
    assert pool.state.tolist() == [len(left), 0] and pool.free[:len(left)].tolist() == left
