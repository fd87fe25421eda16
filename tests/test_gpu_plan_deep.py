"""Trees as deep as prompts are long (tq_kv_plan): chunks given as chains of parents among small trees, and trees
of thousands of rows of any shape. Whole numbers, equal throughout."""

import numpy as np
import pytest
import torch

import rotation_lloyd_max_amd as tq
from test_gpu_plan import check_plan, dev, setup, trees

pytestmark = pytest.mark.gpu


def shapes(n, g):
    """Parents of a tree of n rows, by name."""
    i = np.arange(n)
    chain = np.maximum(i - 1, 0)
    late = chain.copy()
    late[n // 2::97] = np.maximum(i[n // 2::97] - 60, 0)
    broken = chain.copy()
    broken[n - 5] = -1
    first = chain.copy()
    first[1:3] = 0
    return dict(chain=chain, two=np.maximum(i - 2, 0), late=late, broken=broken, first=first, root=np.zeros(n, int),
                far=np.array([0] + [int(g.integers(0, k)) for k in range(1, n)]),
                near=np.array([0] + [int(g.integers(max(0, k - 3), k)) for k in range(1, n)]),
                none=np.where(g.random(n) < 0.01, -1, chain), self=np.where(i % 500 == 499, i, chain))


@pytest.mark.parametrize("shape", ["chain", "two", "late", "broken", "first", "root", "far", "near", "none", "self"])
@pytest.mark.parametrize("n,words", [(256, 9), (257, 8), (513, 17), (2049, 65), (2305, 3), (2600, 0), (4000, 125), (4096, 1)])
def test_deep_trees_among_small_ones(shape, n, words):
    g = np.random.default_rng([n, words])
    counts = [24, n, 3, 0, 700, n - 1, 9]
    lens = [7, 100, 0, 50, 33, 64, 1]
    table, free = setup(g, lens, 64, 300, 90)
    t = [trees(g, [c]) for c in counts]
    t[1], t[5] = shapes(n, g)[shape], shapes(n - 1, g)[shape]
    parents = np.concatenate(t + [[0, 0]]).astype(np.int64)
    shift = g.integers(-99, 99, 7)
    check_plan(lens, counts, table, free, sum(counts) + 2, 64, 300, parents, words, shift)
    # the second of the deep ones is refused, for rows or pages
    check_plan(lens, counts, table, free, sum(counts) - 12, 64, 300, parents[:sum(counts) - 12], words)
    check_plan(lens, counts, table, free[:n // 64 + 15], sum(counts), 64, 300, parents[:-2], words)


def depths(parents):
    d = np.zeros(len(parents), np.int64)
    for i, up in enumerate(parents.tolist()):
        if 0 <= up < i:
            d[i] = d[up] + 1
    return d


def masks(parents, words):
    """By rows, from the ancestors': uint32 [n, words]."""
    m = np.zeros((len(parents), words), np.uint32)
    for i, up in enumerate(parents.tolist()):
        if 0 <= up < i:
            m[i] = m[up]
        if i < 32 * words:
            m[i, i >> 5] |= np.uint32(1 << (i & 31))
    return m


@pytest.mark.parametrize("shape", ["chain", "two", "late", "far", "none"])
@pytest.mark.parametrize("n,words", [(300001, 0), (70000, 40)])
def test_very_deep_trees(shape, n, words):
    g = np.random.default_rng(n)
    parents = shapes(n, g)[shape]
    page, pages = 256, n // 256 + 10
    pool = tq.kv_pool(pages)
    table = torch.full((2, pages), -1, dtype=torch.int32, device="cuda")
    whole = np.concatenate([[0, 0, 1], parents])
    p = tq.kv_plan(pool, dev([0, 0]), dev([3, n]), table, n + 3, page, parents=dev(whole), tree_words=words, shift=dev([0, 7]))
    torch.cuda.synchronize()
    assert p.status.tolist() == [0, 0] and p.kv_lens.tolist() == [3, n]
    assert np.array_equal(p.positions[3:].cpu().numpy(), 7 + depths(parents))
    token = np.arange(n)
    slots = table[1].cpu().numpy()[token // page].astype(np.int64) * page + token % page
    assert np.array_equal(p.slots[3:].cpu().numpy(), slots)
    if words:
        assert np.array_equal(p.tree[3:].cpu().numpy().view(np.uint32), masks(parents, words))


def test_many_deep_trees():
    # more sequences than a workgroup looks at in one go, deep ones in both halves
    g = np.random.default_rng(3)
    B, n = 1100, 2100
    counts = g.integers(0, 3, B)
    counts[[5, 6, 1023, 1024, 1099]] = n
    lens = g.integers(0, 40, B)
    table, free = setup(g, lens, 64, 4000, 40)
    t = [shapes(c, g)[("far", "two", "chain")[b % 3]] if c == n else np.zeros(c, int) for b, c in enumerate(counts)]
    check_plan(lens, counts, table, free, int(counts.sum()), 64, 4000, np.concatenate(t).astype(np.int64), 3)


def test_deep_trees_captured_and_replayed():
    # lengths, rows and parents change between the replays
    B, M, words, page = 6, 5000, 40, 16
    g = np.random.default_rng(8)
    pool, table = tq.kv_pool(500), torch.full((B, 400), -1, dtype=torch.int32, device="cuda")
    z = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    lens, counts, parents, left = z(B), z(B), z(M), z(1)
    call = lambda: tq.kv_plan(pool, lens, counts, table, M, page, parents=parents, tree_words=words, left=left)  # noqa: E731
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p = call()
    for turn, (deep, shape) in enumerate(((1300, "far"), (24, "near"), (4000, "chain"), (2000, "two"), (3000, "late"))):
        n = np.array([5, deep, 0, 24, 300, 9])
        counts.copy_(dev(n))
        lens.zero_()
        parents.zero_()
        parents[:n.sum()] = dev(np.concatenate([shapes(deep, g)[shape] if x == deep else trees(g, [x]) for x in n]))
        graph.replay()
        eager = call()
        torch.cuda.synchronize()
        for x, y in zip(p, eager):
            assert torch.equal(x, y), turn
        d = depths(parents[5:5 + deep].cpu().numpy())
        assert np.array_equal(p.positions[5:5 + deep].cpu().numpy(), d) and p.status.tolist() == [0] * B
