"""Verification of drafted tokens on the GPU against the oracle: whole numbers, equal wherever the oracle's
decisions are clear.

A test of a drafted token compares numbers made with fp32 sums of exponentials 2^t, t = (x - ref) c. The
difference, c and the product are off by half a step (2^-24) each, so t is by 3 2^-24 |t| and 2^t by 3 ln 2 2^-24 |t|;
2^t itself by a step (2^-23), three fp32 additions by 2^-24 each. The kernel keeps |t| below 100 for what counts: together
213 2^-24 = 1.3e-5, for p and for q: 2.6e-5 of what is compared.

The new token's border in the cumulative sum is made with fp64: an exponential is off by 2e-14 of itself plus
2^-52 |t| (t below 1000), sums of n terms by log2(n) + 16 roundings where they are joined pairwise and by n / 256 for
a thread's own, all 2^-53: together below 1e-12 of the sum of w, divided by how much of p + a q is left in it.

The oracle returns each sequence's smallest relative distances to its borders; below these bounds either
side is right, and the sequence is not compared.
"""

import ctypes

import numpy as np
import pytest
import torch

import rotation_lloyd_max_amd as tq
from oracle import step as ost
from parity import as_f64

pytestmark = pytest.mark.gpu
DTS = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
CLEAR = np.array([2.6e-5, 1e-10])     # (a hundredth of p + a q is left in these tests at least)


def case(seed, B, most, V, tdt="bf16", ddt="bf16", kind="logits", tree=False, ragged=True, temperature=None, spread=3.0, noise=0.6,
         hide=0.0):
    """Inputs as a program has them: the draft's values are the target's with noise, drafted tokens
    drawn from its distribution."""
    g = np.random.default_rng([seed, B, most, V])
    counts = g.integers(0, most + 1, B) if ragged else np.full(B, most)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    M = int(offsets[-1])
    parents = np.concatenate([[0] + [int(g.integers(max(0, i - 4), i)) for i in range(1, c)] if c else [] for c in counts]
                             or [[]]).astype(np.int64)
    x = g.standard_normal((M, V)).astype(np.float32) * spread
    y = x + g.standard_normal((M, V)).astype(np.float32) * noise
    if hide:
        gone = g.random((M, V)) < hide
        gone[np.arange(M), g.integers(0, V, M)] = False
        x, y = np.where(gone, -np.inf, x).astype(np.float32), np.where(gone, -np.inf, y).astype(np.float32)
    if kind == "probabilities":
        x, y = (torch.softmax(torch.from_numpy(z), -1).numpy() if M else z for z in (x, y))
    t = torch.from_numpy(x).to(DTS[tdt])
    d = None if ddt is None else torch.from_numpy(y).to(DTS[ddt])
    tokens = np.zeros(M, np.int64)
    src = y if d is None else as_f64(d)
    for b in range(B):
        for i in range(1, counts[b]):
            up = offsets[b] + (parents[offsets[b] + i] if tree else i - 1)
            z = np.log(np.maximum(src[up], 1e-300)) if kind == "probabilities" else src[up] / 1.0
            tokens[offsets[b] + i] = np.argmax(z + g.gumbel(size=V))
    u = g.random(M).astype(np.float32)
    if isinstance(temperature, str):
        temperature = g.random(B).astype(np.float32) * 0.8 + 0.5
        temperature[::3] = 0.0
    return dict(target=t, tokens=tokens, uniforms=u, offsets=offsets, draft=d, parents=parents if tree else None,
                temperature=temperature, target_kind=kind, draft_kind=kind)


def on_gpu(c):
    put = lambda x, dt: None if x is None else torch.as_tensor(x).to(dt).cuda()  # noqa: E731
    t = lambda x: None if x is None else x if x.is_cuda else x.cuda()  # noqa: E731
    return dict(target=t(c["target"]), tokens=put(c["tokens"], torch.int32), uniforms=put(c["uniforms"], torch.float32),
                offsets=put(c["offsets"], torch.int32), draft=t(c["draft"]), parents=put(c["parents"], torch.int32),
                temperature=put(c["temperature"], torch.float32), target_kind=c["target_kind"], draft_kind=c["draft_kind"])


def reference(c):
    f = lambda x: None if x is None else as_f64(x)  # noqa: E731
    return ost.verify(**{**c, "target": f(c["target"]), "draft": f(c["draft"]),
                         "uniforms": np.asarray(c["uniforms"], np.float32).astype(np.float64),
                         "temperature": None if c["temperature"] is None else np.asarray(c["temperature"], np.float32)})


def compare(got, want, offsets, share=0.9):
    """got equal to want for the sequences whose decisions are clear, `share` of them at least."""
    kept, tokens, path, margins = want
    clear = (margins > CLEAR).all(1)
    assert clear.sum() >= share * len(clear) or len(clear) < 3, "the inputs of this test leave decisions open"
    g = [x.cpu().numpy() for x in got]
    assert np.array_equal(g[0][clear], kept[clear]), (g[0], kept)
    rows = np.zeros(len(tokens), bool)
    for b in np.nonzero(clear)[0]:
        rows[offsets[b]:offsets[b + 1]] = True
    assert np.array_equal(g[2][rows], path[rows])
    assert np.array_equal(g[1][rows], tokens[rows]), (g[1], tokens)


def check(c, got=None):
    want = reference(c)
    if got is None:
        got = tq.verify(**on_gpu(c))
    torch.cuda.synchronize()
    compare(got, want, c["offsets"])
    return got


@pytest.mark.parametrize("tdt,ddt", [("bf16", "bf16"), ("fp32", "fp16"), ("fp16", None), ("bf16", "fp32"), ("fp32", None)])
@pytest.mark.parametrize("kind", ["logits", "probabilities"])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("V", [1, 2, 7, 64, 255, 257, 2049, 10007])
def test_matches_oracle(tdt, ddt, kind, tree, V):
    check(case(1, 9, 9, V, tdt, ddt, kind, tree, temperature="mixed"))
    check(case(2, 5, 13, V, tdt, ddt, kind, tree, noise=2.5))


@pytest.mark.parametrize("V", [8191, 8192, 16385, 50257, 131072, 262147])
@pytest.mark.parametrize("tree,ddt", [(False, "bf16"), (True, "fp16"), (True, None)])
def test_large_vocabularies(V, tree, ddt):
    check(case(3, 3, 6, V, "bf16", ddt, "logits", tree, temperature=np.array([0.7, 1.0, 1.3], np.float32)))
    check(case(4, 1, 1, V, "fp32", ddt, "logits", tree))
    check(case(5, 2, 5, V, "fp32", ddt, "probabilities", tree, ragged=False))


def test_many_sequences_and_long_chains():
    check(case(6, 300, 4, 500, noise=0.1))
    check(case(7, 130, 3, 4001, "fp16", None))
    check(case(8, 2, 300, 300, noise=0.02, ragged=False))
    check(case(9, 2, 300, 300, "fp32", None, tree=True, ragged=False, spread=12.0))
    check(case(10, 1, 200, 1000, tree=True, noise=0.05, ragged=False))


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("ddt", ["bf16", None])
def test_masked_vocabularies(tree, ddt):
    # logits of -inf nearly everywhere, whole first and last pieces among them
    check(case(11, 6, 6, 5003, "bf16", ddt, tree=tree, hide=0.99))
    c = case(12, 4, 5, 40000, "fp32", "fp32" if ddt else None, tree=tree)
    for t in (c["target"], c["draft"]):
        if t is not None:
            t[:, :33000] = -np.inf
            t[:, 39000:] = -np.inf
    c["tokens"] = np.where(c["tokens"] < 33000, 33000 + c["tokens"] % 6000, c["tokens"])
    check(c)
    c["target"][:, 33000:38999] = -np.inf       # one token is left
    c["tokens"][1::2] = 38999
    got = check(c)
    end, kept = c["offsets"], got.kept.tolist()
    assert all(got.tokens[end[b] + k - 1].item() == 38999 for b, k in enumerate(kept) if k)


def test_values_of_any_size():
    for dt, big in (("fp32", 3e38), ("bf16", 3e38), ("fp16", 65504.0)):
        c = case(13, 6, 5, 300, dt, dt, temperature=np.array([1.0, 1e30, 0.3, 1e-3, 100.0, 1.0], np.float32))
        c["target"][::2, 100:103] = big
        c["target"][1::2] *= 1000.0
        c["draft"][::3] *= 500.0
        c["target"][2] = -c["target"][2].abs() * 100.0 - 5000.0
        check(c)     # (three equal largest values: thirds, which u meets only by chance)


@pytest.mark.parametrize("T", [0.0, -1.0, float("nan"), float("inf"), 1e-38, 1e-44, 1e38])
def test_temperatures(T):
    for ddt in ("fp16", None):
        c = case(14, 5, 6, 777, "fp16", ddt, temperature=np.full(5, T, np.float32), noise=0.2)
        check(c)
        c["target"][:, 5:500] = -np.inf
        check(c)
    c = case(15, 5, 6, 777, "fp32", "fp32", "probabilities", temperature=np.full(5, T, np.float32))
    check(c)


def test_greedy_takes_the_first_of_equal_values_whatever_the_numbers():
    c = case(16, 6, 7, 3000, "bf16", "bf16", spread=0.3, temperature=np.zeros(6, np.float32))    # many equal values in bf16
    c["target"] = torch.round(c["target"].float() * 2).to(torch.bfloat16)
    for r in range(0, len(c["tokens"]) - 1, 2):
        c["tokens"][r + 1] = int(np.argmax(as_f64(c["target"])[r]))
    check(c)
    for u in (1.0, float("nan"), -3.0):
        c["uniforms"][:] = u
        check(c)


def test_rows_that_are_no_distribution():
    for bad in (float("nan"), float("inf")):
        for where in ("target", "draft"):
            for place in (0, 1500, 2999):
                for T in (None, np.array([0.8, 0.0, 1.0, 0.0, 1.2], np.float32)):
                    c = case(17, 5, 4, 3000, "fp32", "bf16", noise=0.01, ragged=False, temperature=T)
                    c[where][1::3, place] = bad
                    check(c)
    c = case(18, 5, 4, 3000, "fp32", "bf16", noise=0.01, ragged=False)
    c["target"][5] = -np.inf
    c["draft"][8] = -np.inf
    got = check(c)
    assert (got.tokens == -1).sum() > 0
    # probabilities: of the row that the new token comes from
    for bad in (float("nan"), float("inf")):
        c = case(19, 4, 1, 3000, "fp32", None, "probabilities", ragged=False)
        c["target"][2, 777] = bad
        c["target"][3] = 0.0
        got = check(c)
        assert got.tokens.tolist()[2:] == [-1, -1]


def test_numbers_at_their_ends():
    c = case(20, 8, 4, 1200, "fp32", "fp32", ragged=False)
    for u in (0.0, 1.0 - 2.0 ** -24):
        c["uniforms"][:] = u
        check(c)
    # beyond the ends: nothing is accepted, the last token with weight; below: all, the first
    for kind in ("logits", "probabilities"):
        c = case(21, 8, 4, 1200, "fp32", "fp32", kind, ragged=False, hide=0.3 if kind == "logits" else 0.0)
        for u in (1.0, 2.0, float("nan"), -1.0):
            c["uniforms"][:] = u
            got = tq.verify(**on_gpu(c))
            kept, tokens, path, _ = reference(c)
            torch.cuda.synchronize()
            assert np.array_equal(got.kept.cpu().numpy(), kept) and np.array_equal(got.path.cpu().numpy(), path)


def test_nothing_left_falls_back_to_the_target():
    # equal distributions whose tokens are turned away by u = 1, and a point mass turned away
    c = case(22, 4, 2, 50, "fp32", "fp32", ragged=False, noise=0.0)
    c["uniforms"][1::2] = 1.0
    check(c)
    c = case(23, 3, 2, 50, "fp32", None, "probabilities", ragged=False)
    c["target"][:] = 0.0
    c["target"][:, 7] = 1.0
    c["tokens"][:] = 7
    c["uniforms"][1::2] = 1.0
    got = check(c)
    assert got.kept.tolist() == [1, 1, 1] and got.tokens[::2].tolist() == [7, 7, 7]


def test_padding_duplicates_and_parents_that_are_none():
    for ddt in ("bf16", None):
        c = case(24, 6, 9, 40, "bf16", ddt, tree=True, spread=1.0, ragged=False)
        c["tokens"][3::5] = -1
        c["tokens"][4::7] = 40
        c["tokens"][1::9] = c["tokens"][2::9]
        c["parents"][2::9] = c["parents"][1::9] = 0
        c["parents"][5::9] = 7
        c["parents"][6::9] = -1
        check(c)
        c["parents"][:] = 0          # eight children of the root, few tokens: the same one several times
        check(c)


@pytest.mark.parametrize("tdt,ddt", [("bf16", "fp16"), ("fp32", "bf16"), ("fp16", "fp32")])
def test_strides_and_odd_addresses(tdt, ddt):
    c = case(25, 5, 5, 4097, tdt, ddt)
    g = on_gpu(c)
    for shift in (0, 1, 3):
        for name in ("target", "draft"):
            t = c[name]
            wide = torch.full((t.shape[0], t.shape[1] + 5 + shift), float("nan"), dtype=t.dtype, device="cuda")
            wide[:, shift:shift + t.shape[1]] = t.cuda()
            g[name] = wide[:, shift:shift + t.shape[1]]
        check(c, tq.verify(**g))
    one = on_gpu(case(26, 3, 1, 1000, tdt, None, ragged=False))
    one["target"] = one["target"][:1].expand(3, -1)       # one row for every sequence
    got = tq.verify(**one)
    assert got.kept.tolist() == [1, 1, 1]


def test_rows_behind_the_last_sequence_are_left():
    c = case(27, 4, 5, 600, ragged=False)
    g = on_gpu(c)
    g["offsets"][2:] -= 3
    M = 20
    out = [torch.full((n,), 1234, dtype=torch.int32, device="cuda") for n in (4, M, M)]
    need = tq.verify_workspace(600, 4, M, True)
    ws = torch.empty(max(1, need), dtype=torch.uint8, device="cuda")
    rc = tq.lib().tq_verify(g["target"].data_ptr(), tq.BF16, 600, g["draft"].data_ptr(), tq.BF16, 600, 0, 600, 4,
                            g["offsets"].data_ptr(), M, g["tokens"].data_ptr(), None, g["uniforms"].data_ptr(), None,
                            out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), ws.data_ptr(), need,
                            torch.cuda.current_stream().cuda_stream)
    assert rc == 0, tq.lib().tq_last_error()
    torch.cuda.synchronize()
    assert (out[1][17:] == 1234).all() and (out[2][17:] == 1234).all() and not (out[1][:17] == 1234).any()
    c["offsets"] = g["offsets"].cpu().numpy()
    kept, tokens, path, _ = reference(c)
    assert np.array_equal(out[0].cpu().numpy(), kept) and np.array_equal(out[1][:17].cpu().numpy(), tokens[:17])


def test_no_rows():
    e = torch.empty
    for B in (0, 3):
        got = tq.verify(e((0, 100), device="cuda"), e(0, dtype=torch.int32, device="cuda"), e(0, device="cuda"),
                        torch.zeros(B + 1, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        assert got.kept.tolist() == [0] * B


def test_repeated_calls_streams_and_graphs():
    # replays over new inputs, two graphs and eager calls in turn, each with a workspace of its own
    cs = [case(s, 7, 6, 9001, "bf16", "bf16" if s % 2 else None, tree=s > 29) for s in (28, 29, 30, 31)]
    gs = [on_gpu(c) for c in cs]
    want = [check(c) for c in cs]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        other = [tq.verify(**g) for g in gs]
    st.synchronize()
    for a, b, c in zip(want, other, cs):
        end = int(c["offsets"][-1])
        assert torch.equal(a.kept, b.kept) and torch.equal(a.tokens[:end], b.tokens[:end])
    graphs, outs = [], []
    for g in gs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(tq.verify(**g))
        graphs.append(graph)
    for turn in range(3):
        for g in gs:
            g["uniforms"].copy_(torch.rand_like(g["uniforms"]))
        for graph, g, o in zip(graphs, gs, outs):
            graph.replay()
            eager = tq.verify(**g)
            torch.cuda.synchronize()
            end = g["offsets"][-1].item()
            assert torch.equal(o.kept, eager.kept) and torch.equal(o.tokens[:end], eager.tokens[:end])
            assert torch.equal(o.path[:end], eager.path[:end])


def test_frequencies_follow_the_target():
    # 4000 sequences over one pair of distributions: counts of the first new token against p, each within
    # five standard deviations of its binomial count
    g = np.random.default_rng(33)
    V, n = 24, 4000
    x, y = g.standard_normal(V) * 1.5, g.standard_normal(V) * 1.5
    p, q = (np.exp(z) / np.exp(z).sum() for z in (x, y))
    for parents, rows in ((None, 2), (np.tile([0, 0, 0, 0], n), 4)):
        tokens = np.zeros((n, rows), np.int64)
        tokens[:, 1:] = g.choice(V, (n, rows - 1), p=q)
        put = lambda z: torch.from_numpy(z.astype(np.float32)).cuda().expand(n * rows, -1)  # noqa: E731
        got = tq.verify(put(x), torch.from_numpy(tokens.reshape(-1)).cuda(),
                        torch.from_numpy(g.random(n * rows).astype(np.float32)).cuda(),
                        torch.arange(0, n * rows + 1, rows, device="cuda"), draft=put(y),
                        parents=None if parents is None else torch.from_numpy(parents).cuda())
        first = np.bincount(got.tokens.view(n, rows)[:, 0].cpu().numpy(), minlength=V)
        assert np.all(np.abs(first - n * p) <= 5 * np.sqrt(n * p * (1 - p)) + 1)


@pytest.mark.parametrize("ddt", ["fp32", None])
def test_broad_trees_of_many_rows(ddt):
    # three children to a row, 700 rows: accepted rows beyond the first 256, siblings turned away on the way there
    c = case(34, 16, 700, 60, "fp32", ddt, ragged=False, noise=0.5, spread=1.5 if ddt else 5.0)
    n = 700
    up = np.concatenate([[0], (np.arange(1, n) - 1) // 3])
    c["parents"] = np.tile(up, 16)
    g = np.random.default_rng(35)
    src = as_f64(c["target"] if ddt is None else c["draft"])
    for r in range(16 * n):
        if r % n:
            c["tokens"][r] = np.argmax(src[r - r % n + up[r % n]] + g.gumbel(size=60))
    if ddt is None:
        c["uniforms"] *= 0.5           # (point masses stay as often as their probability says)
    got = check(c)
    path = got.path.view(16, n).cpu().numpy()
    assert (path.max(1) >= 256).sum() >= 4
    later = [(path[b, i] - 1) % 3 for b in range(16) for i in range(1, got.kept[b].item())]
    assert any(later), "no sibling was turned away"


@pytest.mark.parametrize("ddt", ["fp32", "bf16", None])
def test_many_children_of_one_row(ddt):
    # all rows are the root's children, more than LDS holds, some tokens twice; nearly all are turned away
    for n, V in ((13, 500), (300, 5000), (700, 20001)):
        c = case(36, 6, n, V, "fp32", ddt, ragged=False, noise=2.0, spread=1.0)
        c["parents"] = np.zeros(6 * n, np.int64)
        g = np.random.default_rng([37, n])
        src = as_f64(c["target"] if ddt is None else c["draft"])
        for r in range(6 * n):
            c["tokens"][r] = np.argmax(src[r - r % n] + g.gumbel(size=V))
        if ddt is not None:     # the first eight are tokens that the draft likes far more than the target
            for b in range(6):
                c["tokens"][b * n + 1:b * n + 9] = np.argsort(as_f64(c["target"])[b * n] - src[b * n])[:8]
        c["tokens"][3::n] = c["tokens"][2::n]
        c["uniforms"] = (1.0 - c["uniforms"] * (1e-3 if ddt is None else 0.03)).astype(np.float32)
        check(c)


@pytest.mark.parametrize("T", [1e-44, 1e-6, 1e38, float("inf")])
def test_siblings_at_extreme_temperatures(T):
    for tdt in ("fp32", "bf16"):
        c = case(38, 6, 9, 777, tdt, tdt, tree=True, temperature=np.full(6, T, np.float32), noise=1.0, ragged=False)
        c["parents"][:] = np.tile([0, 0, 0, 0, 1, 1, 2, 2, 2], 6)
        check(c)
        c["target"][:, 5:500] = -np.inf
        check(c)


@pytest.mark.parametrize("tree,ddt", [(False, "bf16"), (True, "fp32"), (True, None)])
def test_more_pieces_of_a_row_than_lanes_hold(tree, ddt):
    # above 64 pieces of 8192 tokens
    for kind in ("logits", "probabilities"):
        check(case(39, 2, 4, 600001, "fp32", ddt, kind, tree, ragged=False, noise=1.5))
    check(case(40, 2, 3, 1100000, "bf16", ddt, "logits", tree, ragged=False, temperature=np.array([0.0, 0.9], np.float32)))


@pytest.mark.parametrize("ddt", ["fp32", None])
def test_long_chains_that_end_anywhere(ddt):
    # 64 rows are looked at at once, 256 are in LDS: all stay, one is turned away or is padding near the ends of these
    n = 600
    c = case(41, 12, n, 40, "fp32", ddt, ragged=False, noise=0.0, spread=2.0)
    c["uniforms"] = (c["uniforms"] * 1e-4).astype(np.float32)
    src = as_f64(c["target"])
    c["tokens"] = np.concatenate([[0], np.argmax(src[:-1], 1)])       # the likeliest tokens: all stay
    if ddt:
        c["draft"] = c["target"].clone()
    ends = (0, 1, 63, 64, 65, 127, 255, 256, 257, 511, 598, 599)
    for b, e in enumerate(ends):
        row = b * n + e + 1
        if e + 1 < n:
            if b % 2:
                c["tokens"][row] = -1
            else:
                c["uniforms"][row] = 1.0
                if ddt is None:
                    c["tokens"][row] = np.argmin(src[row - 1])
    got = check(c)
    assert got.kept.tolist() == [e + 1 for e in ends]


def test_rows_gigabytes_apart():
    c = case(42, 2, 3, 5000, "bf16", "fp32", ragged=False)
    g = on_gpu(c)
    for name in ("target", "draft"):
        t = g[name]
        wide = torch.empty(5 * (1 << 30) + 5000, dtype=t.dtype, device="cuda").as_strided((6, 5000), (1 << 30, 1))
        wide.copy_(t)
        g[name] = wide
    check(c, tq.verify(**g))


@pytest.mark.parametrize("ddt", ["bf16", None])
def test_as_many_sequences_as_there_may_be(ddt):
    check(case(43, 65536, 2, 5, "bf16", ddt))
    check(case(44, 3000, 3, 130, "fp16", ddt, tree=True, temperature="mixed"))


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("kinds", [("logits", "probabilities"), ("probabilities", "logits")])
@pytest.mark.parametrize("tdt,ddt", [("bf16", "fp32"), ("fp32", "fp32"), ("fp16", "bf16")])
def test_logits_against_probabilities(tdt, ddt, kinds, tree):
    for seed, V in ((45, 100), (46, 5000)):
        c = case(seed, 9, 9, V, tdt, ddt, tree=tree, noise=1.5, temperature="mixed")
        for name, kind, dt in zip(("target", "draft"), kinds, (tdt, ddt)):
            c[name + "_kind"] = kind
            if kind == "probabilities":
                c[name] = torch.softmax(c[name].float(), -1).to(DTS[dt])
        check(c)


@pytest.mark.parametrize("kind,dt", [("logits", "fp32"), ("logits", "bf16"), ("probabilities", "fp32")])
@pytest.mark.parametrize("gone", [1, 2, 3, 4, 5])
def test_little_left_after_siblings_the_draft_would_hardly_draw(kind, dt, gone):
    # one token has nearly all of p and of q: each other sibling leaves a fortieth of S, 1e-8 after the last
    B, V, n = 64, 300, gone + 3
    c = case(47 + gone, B, n, V, "fp32", "fp32", ragged=False, tree=True, spread=0.5, noise=0.1)
    c["parents"] = np.zeros(B * n, np.int64)
    c["target"][:, 7], c["draft"][:, 7] = 10.4, 9.6
    for name in ("target", "draft"):
        if kind == "probabilities":
            c[name] = torch.softmax(c[name].double(), -1).float()
        c[name] = c[name].to(DTS[dt])
        c[name + "_kind"] = kind
    p, q = (ost.distribution(as_f64(c[x])[0], kind, 1.0) for x in ("target", "draft"))
    assert p[7] > q[7] > 0.97
    for b in range(B):
        p, q = (ost.distribution(as_f64(c[x])[b * n], kind, 1.0) for x in ("target", "draft"))
        c["tokens"][b * n + 1:b * n + 1 + gone] = np.argsort(p / q)[:gone]       # none of these stays
    c["tokens"][1 + gone::n] = 7
    c["uniforms"][1::n] = 0.999
    c["uniforms"][1 + gone::n] = np.linspace(0.9, 1.1, B)
    got = check(c)
    assert (got.kept == 2).sum() > B // 4 and (got.kept == 1).sum() > B // 16
