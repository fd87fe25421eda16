"""The oracle of a decoding step against the properties that define it: verified tokens are distributed
as the target's, pages are neither lost nor given twice."""

import numpy as np
import pytest

from oracle import step as ost


def grid(n):
    """n numbers whose mean of a step function is off by at most 1 / (2 n) per step."""
    return (np.arange(n) + 0.5) / n


P = np.array([0.4, 0.05, 0.3, 0.0, 0.25])
Q = np.array([0.1, 0.5, 0.2, 0.2, 0.0])


def new_tokens(tokens, parents, uniforms, draft, seqs):
    n = len(tokens)
    target = np.tile(P, (n, 1))
    kept, out, path, _ = ost.verify(target, tokens, uniforms, [0, n], draft, parents, None, "probabilities", "probabilities")
    return int(out[0])


def test_one_draft_keeps_the_targets_distribution():
    # the token x is drawn from q; accepted or replaced, the first new token is distributed as p
    u, freq = grid(40), np.zeros(5)
    for x in range(5):
        for u0 in u:
            for u1 in u:
                first = new_tokens([0, x], None, [u0, u1], np.tile(Q, (2, 1)), 1)
                freq[first] += Q[x] / u.size ** 2
    np.testing.assert_allclose(freq, P, atol=6 / 40)
    assert abs(freq.sum() - 1.0) < 1e-12


def test_siblings_keep_the_targets_distribution():
    u, freq = grid(12), np.zeros(5)
    for x in range(5):
        for y in range(5):
            if Q[x] * Q[y] == 0.0:
                continue
            for u0 in u:
                for u1 in u:
                    for u2 in u:
                        first = new_tokens([0, x, y], [0, 0, 0], [u0, u1, u2], np.tile(Q, (3, 1)), 1)
                        freq[first] += Q[x] * Q[y] / u.size ** 3
    np.testing.assert_allclose(freq, P, atol=0.09)     # three grids of 12: each decision off by at most 1 / 24


@pytest.mark.parametrize("children", [[2], [2, 0], [1, 1, 4], [0, 1, 2, 4]])
def test_fixed_drafts_keep_the_targets_distribution(children):
    u, freq = grid(8), np.zeros(5)
    n = len(children)
    for k in range(8 ** (n + 1)):
        pick = [u[(k // 8 ** i) % 8] for i in range(n + 1)]
        freq[new_tokens([0] + children, [0] * (n + 1), pick, None, 1)] += 1 / 8 ** (n + 1)
    np.testing.assert_allclose(freq, P, atol=(n + 1) / 16)


def test_recursion_of_what_is_left():
    # (p - a q)+ with a growing by its sum is the renormalised left-over, step after step
    g = np.random.default_rng(3)
    for _ in range(20):
        p, q = g.dirichlet(np.ones(30) * 0.3), g.dirichlet(np.ones(30) * 0.3)
        left, a, S = p, 0.0, 1.0
        for _ in range(6):
            a += S
            S = np.maximum(p - a * q, 0).sum()
            left = np.maximum(left - q, 0)
            if left.sum() == 0.0:
                assert S < 1e-12
                break
            left /= left.sum()
            np.testing.assert_allclose(np.maximum(p - a * q, 0) / S, left, atol=1e-9)


def test_pages_are_conserved():
    g = np.random.default_rng(5)
    pages, page, B, width = 40, 16, 5, 9
    free, table, lens = list(range(pages)), np.full((B, width), -1), np.zeros(B, int)
    for step in range(60):
        counts = g.integers(0, 30, B)
        p = ost.plan(free, lens, counts, table, 200, page, pages)
        held = [int(x) for b in range(B) for x in p["table"][b][:-(-max(p["kv_lens"][b], 0 if p["status"][b] == 0 else lens[b]) // page)]]
        assert sorted(held + p["free"]) == list(range(pages))
        slots = p["slots"][p["slots"] >= 0]
        assert np.unique(slots).size == slots.size
        kept = np.array([g.integers(0, c + 1) if g.random() < 0.9 else -1 for c in counts])
        lens, free, _ = ost.keep(p["free"], lens, kept, p["table"], page, p["q_offsets"], p["status"])
        table = p["table"]
        held = [int(x) for b in range(B) for x in table[b][:-(-lens[b] // page)]]
        assert sorted(held + free) == list(range(pages))


def test_keeping_nothing_undoes_the_plan():
    free, table, lens = list(range(20)), np.full((3, 6), -1), np.array([17, 0, 33])
    p = ost.plan(free, lens, [40, 3, 1], table, 44, 16, 20)
    assert len(p["free"]) < 20
    ends, back, _ = ost.keep(p["free"], lens, [0, 0, 0], p["table"], 16, p["q_offsets"], p["status"])
    assert back == free and list(ends) == list(lens)
