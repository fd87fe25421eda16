"""Decoding steps with drafted tokens as a program runs them: plan, turn, store, attend, verify, keep, nothing
read on the host in between. A small "model" (embeddings, one layer of attention, a projection) gives the
logits. After every step the caches hold, byte for byte, what storing the accepted texts token by token
into a fresh cache gives, and lengths, pages and tokens are the oracle's."""

import numpy as np
import pytest
import torch

import rotation_lloyd_max_amd as tq
from oracle import step as ost
from parity import as_f64
from test_gpu_verify import CLEAR

pytestmark = pytest.mark.gpu
V, HEADS, SHARE, D, PAGE, WIDTH = 97, 2, 2, 64, 16, 12
SECTIONS = (8, 12, 12)


class Model:
    def __init__(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.q, self.k, self.v = r(V, HEADS * SHARE, D).bfloat16(), r(V, HEADS, D).bfloat16(), r(V, HEADS, D).bfloat16()
        self.head = (r(V, HEADS * SHARE * D) * 0.05).bfloat16()
        self.guess = r(V, V) * 1.5
        self.rope = tq.rope_axes(SECTIONS)


class Batch:
    """What a serving program keeps: the cache, pages, tables, lengths, and the step's inputs."""

    def __init__(self, model, B, rows, pages, words, draft, seed):
        self.m, self.B, self.rows, self.words = model, B, rows, words
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.cache = tq.kv_cache(pages, HEADS, D, page_tokens=PAGE)
        self.pool = tq.kv_pool(pages)
        self.table = torch.full((B, WIDTH), -1, dtype=torch.int32, device="cuda")
        z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
        self.lens, self.counts, self.tokens, self.parents = z(B), z(B), z(rows), z(rows)
        self.uniforms, self.temperature = z(rows, dt=torch.float32), torch.full((B,), 0.9, device="cuda")
        self.temperature[-1] = 0.0
        self.axis_shift = torch.arange(3, device="cuda", dtype=torch.int32)[:, None] * 5
        self.draft = draft

    def step(self):
        m = self.m
        p = tq.kv_plan(self.pool, self.lens, self.counts, self.table, self.rows, PAGE, parents=self.parents,
                       tree_words=self.words)
        tok = self.tokens.long()
        pos = p.positions + self.axis_shift
        q = tq.rope(m.q[tok], pos, m.rope)
        tq.kv_store(self.cache, m.k[tok], m.v[tok], p.slots, rope=m.rope, positions=pos)
        out = tq.kv_attend(self.cache, q, p.kv_lens, self.table, q_offsets=p.q_offsets, tree=p.tree, out=torch.zeros_like(q))
        logits = (out.view(self.rows, -1) @ m.head.t()).float() + m.guess[tok]
        guess = m.guess[tok] if self.draft else None
        got = tq.verify(logits, self.tokens, self.uniforms, p.q_offsets, draft=guess, parents=self.parents,
                        temperature=self.temperature)
        tq.kv_keep(self.pool, self.lens, got.kept, self.table, PAGE, q_offsets=p.q_offsets, status=p.status, path=got.path,
                   cache=self.cache, out=self.lens)
        return p, logits, got

    def fill(self, roots, most):
        """Drafted trees for the next step, drawn from the guesses (host side of the program)."""
        g = np.random.default_rng(int(torch.randint(1 << 30, (1,), generator=self.g, device="cuda").item()))
        counts = g.integers(1, most + 1, self.B)
        while counts.sum() > self.rows:
            counts[np.argmax(counts)] -= 1
        guess = as_f64(self.m.guess)
        tokens, parents = np.zeros(self.rows, np.int64), np.zeros(self.rows, np.int64)
        at = 0
        for b in range(self.B):
            tokens[at] = roots[b]
            for i in range(1, counts[b]):
                parents[at + i] = g.integers(max(0, i - 3), i)
                T = 1.0 if b == self.B - 1 else 0.9
                tokens[at + i] = np.argmax(guess[tokens[at + parents[at + i]]] / T + g.gumbel(size=V))
            at += counts[b]
        for mine, x in ((self.counts, counts), (self.tokens, tokens), (self.parents, parents), (self.uniforms, g.random(self.rows))):
            mine.copy_(torch.from_numpy(x).to(mine.dtype))
        return counts, tokens, parents


def stored(b, texts):
    """The cache's rows of the texts, from a fresh cache: (key codes, scales, value codes, scales) per text."""
    out = []
    for t in texts:
        n = len(t)
        c = tq.kv_cache(-(-max(1, n) // PAGE), HEADS, D, page_tokens=PAGE)
        tok = torch.tensor(t, device="cuda", dtype=torch.int64)
        pos = torch.arange(n, device="cuda", dtype=torch.int32) + b.axis_shift
        tq.kv_store(c, b.m.k[tok], b.m.v[tok], torch.arange(n, device="cuda"), rope=b.m.rope, positions=pos)
        out.append(rows_of(c, torch.arange(-(-max(1, n) // PAGE), device="cuda"), n))
    return out


def rows_of(cache, pages, n):
    res = []
    for w in (cache.k, cache.v):
        for t in (w.codes, w.scales):
            x = t[pages.long()].view(len(pages), HEADS, PAGE, -1).transpose(1, 2).reshape(len(pages) * PAGE, HEADS, -1)
            res.append(x[:n].clone())
    return res


@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("captured", [False, True])
def test_steps(draft, captured):
    B, most, rows, pages = 5, 9, 36, 9      # (too few for all texts at their longest)
    model = Model(1)
    b = Batch(model, B, rows, pages, 1, draft, 2)
    g = np.random.default_rng(3)
    texts = [[] for _ in range(B)]           # tokens in the cache
    roots = g.integers(0, V, B)
    free, table, lens = list(range(pages - 1, -1, -1)), np.full((B, WIDTH), -1), np.zeros(B, int)
    graph = outs = None
    accepted = refused = 0
    if captured:
        b.fill(roots, most)
        keep = [t.clone() for t in (b.pool.free, b.pool.state, b.table, b.lens)]
        b.step()                             # (warms the library up before the capture)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = b.step()
        for t, k in zip((b.pool.free, b.pool.state, b.table, b.lens), keep):
            t.copy_(k)
    for step in range(24):
        counts, tokens, parents = b.fill(roots, most)
        if captured:
            graph.replay()
            p, logits, got = outs
        else:
            p, logits, got = b.step()
        torch.cuda.synchronize()
        want = ost.plan(free, lens, counts, table, rows, PAGE, pages, parents, 1)
        for name in ("slots", "positions", "q_offsets", "kv_lens", "status"):
            assert np.array_equal(getattr(p, name).cpu().numpy(), want[name]), name
        assert np.array_equal(p.tree.cpu().numpy().view(np.uint32), want["tree"])
        total = int(counts.sum())
        assert not np.isnan(as_f64(logits)[:total]).any()
        T = b.temperature.cpu().numpy()
        kept, new, path, margins = ost.verify(as_f64(logits), tokens, as_f64(b.uniforms), want["q_offsets"],
                                             as_f64(model.guess)[tokens] if draft else None, parents, T)
        assert (margins > CLEAR).all()       # (five sequences, a handful of tests a step)
        assert np.array_equal(got.kept.cpu().numpy(), kept)
        assert np.array_equal(got.tokens.cpu().numpy()[:total], new[:total])
        lens2, free, _ = ost.keep(want["free"], lens, kept, want["table"], PAGE, want["q_offsets"], want["status"])
        table = want["table"]
        assert np.array_equal(b.lens.cpu().numpy(), lens2) and np.array_equal(b.table.cpu().numpy(), table)
        assert b.pool.state.tolist() == [len(free), 0] and b.pool.free[:len(free)].tolist() == free
        for s in range(B):
            lo, k = want["q_offsets"][s], kept[s]
            if want["status"][s]:
                refused += 1
                continue
            texts[s] += [int(roots[s])] + [int(x) for x in new[lo:lo + k - 1]]
            roots[s] = new[lo + k - 1]
            accepted += k - 1
        lens = lens2
        assert [len(t) for t in texts] == list(lens)
        for s, (text, fresh) in enumerate(zip(texts, stored(b, texts))):
            mine = rows_of(b.cache, b.table[s, :-(-max(1, len(text)) // PAGE)].clamp(min=0), len(text))
            assert all(torch.equal(x, y) for x, y in zip(mine, fresh)), (step, s)
        if step in (9, 17):                  # a text ends: its pages come back, another one begins
            end = np.where(np.arange(B) == step % B, -1, 0)
            tq.kv_keep(b.pool, b.lens, torch.from_numpy(end).cuda(), b.table, PAGE, out=b.lens)
            lens, free, _ = ost.keep(free, lens, end, table, PAGE)
            texts[step % B] = []
            torch.cuda.synchronize()
            assert np.array_equal(b.lens.cpu().numpy(), lens)
    assert accepted > 10 and refused > 0


def test_two_batches_captured_and_replayed_in_turn():
    # two graphs, each with its own pool, cache and workspaces, replayed between each other's steps and
    # eager ones, against a batch that runs the same inputs eagerly
    model = Model(4)
    mine = [Batch(model, 4, 20, 40, 1, draft, 5) for draft in (False, True)]
    ref = [Batch(model, 4, 20, 40, 1, draft, 5) for draft in (False, True)]
    graphs = []
    for b in mine:
        b.fill([1, 2, 3, 4], 5)
        state = (b.pool.free, b.pool.state, b.table, b.lens, b.cache.k.codes, b.cache.k.scales, b.cache.v.codes, b.cache.v.scales)
        start = [t.clone() for t in state]
        b.step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = b.step()
        graphs.append((graph, out))
        for t, s in zip(state, start):
            t.copy_(s)
    for step in range(5):
        for b, r, (graph, out) in zip(mine, ref, graphs):
            b.fill([1, 2, 3, 4], 5)
            for name in ("counts", "tokens", "parents", "uniforms"):
                getattr(r, name).copy_(getattr(b, name))
            graph.replay()
            _, _, want = r.step()
            torch.cuda.synchronize()
            n = int(b.counts.sum())
            assert torch.equal(out[2].kept, want.kept) and torch.equal(out[2].tokens[:n], want.tokens[:n])
            assert torch.equal(b.lens, r.lens) and torch.equal(b.pool.state, r.pool.state)
            same = torch.equal(b.cache.k.codes, r.cache.k.codes) and torch.equal(b.cache.v.scales, r.cache.v.scales)
            assert same
