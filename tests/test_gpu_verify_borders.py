"""Decisions of tq_verify close to their borders, against the oracle.

Bounds. Where two numbers are closer than fp32 sums can tell, they are made with fp64 sums: an exponential is off by
2e-14 of itself plus 2^-52 |t| (t below 1000: 2e-13), a sum by 1e-14 of itself; p and q by 4e-13 each, together less
than 1e-12 of what is compared. Without a draft S is 1 less the p of those that went, off by as much of them, so a test
of u S against p is right where they are further apart than 1e-12 (u + p), whatever is left in S.
"""

import numpy as np
import pytest
import torch

import rotation_lloyd_max_amd as tq
from oracle import step as ost
from parity import as_f64
from test_gpu_verify import DTS, case, on_gpu, reference

pytestmark = pytest.mark.gpu


def probabilities(x):
    return np.stack([ost.distribution(r, "logits", 1.0) for r in as_f64(x)])


@pytest.mark.parametrize("dt", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("gone", [2, 4, 7])
def test_little_left_after_fixed_siblings(dt, gone):
    # the likeliest tokens went, 1e-3 or so is left; the next one's number lies at u S = p (1 +- 3e-4), (1 +- 1e-5)
    B, V, n = 512, 700, gone + 2
    c = case(60 + gone, B, n, V, "fp32", None, tree=True, ragged=False, spread=2.0)
    x = c["target"].clone()
    g = np.random.default_rng(61)
    for b in range(B):
        at = g.permutation(V)[:gone]
        x[b * n:(b + 1) * n, at] = torch.from_numpy((15.0 + g.random(gone)).astype(np.float32))
        c["tokens"][b * n + 1:b * n + 1 + gone] = at
    c["target"] = x.to(DTS[dt])
    c["parents"] = np.zeros(B * n, np.int64)
    p = probabilities(c["target"])[::n]
    clear = 0
    for b in range(B):
        at = c["tokens"][b * n + 1:b * n + 1 + gone]
        c["uniforms"][b * n + 1:b * n + 1 + gone] = 1.0 - 2.0 ** -24
        rest = p[b].copy()
        rest[at] = 0.0
        S = rest.sum()
        x = np.argsort(rest)[-1 - b % 40]
        c["tokens"][b * n + n - 1] = x
        u = rest[x] / S * (1.0 + [3e-4, -3e-4, 1e-5, -1e-5][b % 4])
        assert u < 1.0
        c["uniforms"][b * n + n - 1] = u
    kept, tokens, path, _ = reference(c)
    got = tq.verify(**on_gpu(c))
    torch.cuda.synchronize()
    for b in range(B):
        u, t = float(c["uniforms"][b * n + n - 1]), c["tokens"][b * n + n - 1]
        at = c["tokens"][b * n + 1:b * n + 1 + gone]
        S, q = 1.0 - p[b, at].sum(), p[b, t]
        last = float(c["uniforms"][b * n + gone]) * (1.0 - p[b, at[:-1]].sum()) - p[b, at[-1]]
        if abs(u * S - q) > 2e-12 * (u + q) and abs(last) > 2e-12:
            clear += 1
            assert got.kept[b].item() == kept[b], (b, u, S, q)
    assert clear > B // 2


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("tdt,ddt,dkind", [("fp32", "fp32", "logits"), ("bf16", "fp16", "logits"), ("fp32", "bf16", "probabilities"),
                                           ("bf16", None, "logits")])
def test_numbers_next_to_the_border_of_their_test(tdt, ddt, dkind, tree):
    # u is the 32-bit number nearest to p / q (to p without a draft), or a neighbour of it
    B, V = 1500, 900
    c = case(70, B, 3, V, tdt, ddt, tree=tree, ragged=False, spread=4.0)
    c["draft_kind"] = dkind
    if tree:
        c["parents"] = np.tile([0, 0, 0], B)
    p = probabilities(c["target"])[::3]
    if ddt is None:
        q = np.ones_like(p)
    else:
        if dkind == "probabilities":
            c["draft"] = torch.softmax(c["draft"].double(), -1).to(DTS[ddt])
        q = as_f64(c["draft"])[::3] if dkind == "probabilities" else probabilities(c["draft"])[::3]
    likelier = [np.nonzero((p[b] < q[b]) & (p[b] > 1e-9))[0] for b in range(B)]
    at = [int(x[b % x.size]) for b, x in enumerate(likelier)]
    u = np.array([p[b, x] / q[b, x] for b, x in enumerate(at)]).astype(np.float32)
    u[1::3], u[2::3] = np.nextafter(u[1::3], np.float32(0)), np.nextafter(u[2::3], np.float32(2))
    c["tokens"][1::3], c["uniforms"][1::3] = at, np.minimum(u, np.float32(1 - 2.0 ** -24))
    c["uniforms"][2::3] = 1.0 - 2.0 ** -24
    kept, _, path, _ = reference(c)
    got = tq.verify(**on_gpu(c))
    torch.cuda.synchronize()
    first = got.path.view(B, 3)[:, 1].cpu().numpy() == 1
    check_first_tests(c, first, at, p, q, path)


def check_first_tests(c, first, at, p, q, path):
    B, n = len(at), 0
    for b, x in enumerate(at):
        u = float(c["uniforms"][3 * b + 1])
        if abs(u * q[b, x] - p[b, x]) > 1e-12 * (u * q[b, x] + p[b, x]):
            n += 1
            assert first[b] == (u * q[b, x] < p[b, x]) == (path[3 * b + 1] == 1), (b, u, q[b, x], p[b, x])
    assert n > B * 0.98 or n >= B - 1


@pytest.mark.parametrize("tree", [False, True])
def test_probabilities_against_logits_next_to_the_border(tree):
    # the other way round, and captured: replays decide as eager calls do, and alike each time
    B, V = 1500, 900
    c = case(71, B, 3, V, "fp32", "bf16", tree=tree, ragged=False, spread=4.0)
    c["target"] = torch.softmax(c["target"].double(), -1).float()
    c["target_kind"] = "probabilities"
    if tree:
        c["parents"] = np.tile([0, 0, 0], B)
    p, q = as_f64(c["target"])[::3], probabilities(c["draft"])[::3]
    likelier = [np.nonzero((p[b] < q[b]) & (p[b] > 1e-9))[0] for b in range(B)]
    at = [int(x[b % x.size]) for b, x in enumerate(likelier)]
    u = np.array([p[b, x] / q[b, x] for b, x in enumerate(at)]).astype(np.float32)
    u[1::3], u[2::3] = np.nextafter(u[1::3], np.float32(0)), np.nextafter(u[2::3], np.float32(2))
    c["tokens"][1::3], c["uniforms"][1::3] = at, np.minimum(u, np.float32(1 - 2.0 ** -24))
    c["uniforms"][2::3] = 1.0 - 2.0 ** -24
    _, _, path, _ = reference(c)
    g = on_gpu(c)
    eager = tq.verify(**g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replayed = tq.verify(**g)
    for _ in range(4):
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(eager, replayed):
            assert torch.equal(x, y)
    check_first_tests(c, eager.path.view(B, 3)[:, 1].cpu().numpy() == 1, at, p, q, path)


@pytest.mark.parametrize("B,V", [(60, 10007), (8, 131075)])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("tdt,ddt", [("fp32", "bf16"), ("fp16", "fp16"), ("bf16", None)])
def test_large_vocabularies_next_to_the_border(B, V, tdt, ddt, tree):
    c = case(72, B, 3, V, tdt, ddt, tree=tree, ragged=False, spread=4.0, temperature=np.linspace(0.4, 2.5, B).astype(np.float32))
    if tree:
        c["parents"] = np.tile([0, 0, 0], B)
    rows = lambda x: np.stack([ost.distribution(as_f64(x[3 * b:3 * b + 1])[0], "logits", float(c["temperature"][b]))  # noqa: E731
                               for b in range(B)])
    p = rows(c["target"])
    q = np.ones_like(p) if ddt is None else rows(c["draft"])
    likelier = [np.nonzero((p[b] < q[b]) & (p[b] > 1e-12))[0] for b in range(B)]
    at = [int(x[(b * 7919) % x.size]) for b, x in enumerate(likelier)]
    u = np.array([p[b, x] / q[b, x] for b, x in enumerate(at)]).astype(np.float32)
    u[1::3], u[2::3] = np.nextafter(u[1::3], np.float32(0)), np.nextafter(u[2::3], np.float32(2))
    c["tokens"][1::3], c["uniforms"][1::3] = at, np.minimum(u, np.float32(1 - 2.0 ** -24))
    c["uniforms"][2::3] = 1.0 - 2.0 ** -24
    _, _, path, _ = reference(c)
    got = tq.verify(**on_gpu(c))
    torch.cuda.synchronize()
    check_first_tests(c, got.path.view(B, 3)[:, 1].cpu().numpy() == 1, at, p, q, path)


@pytest.mark.parametrize("parents", [None, [0, 0]])
def test_rows_that_differ_in_two_tokens(parents):
    # p and q are alike but for a token that p likes more and one that it likes less, by as much but for 1e-9 to 1e-6
    # of the whole: the many tokens in between have w = p - q of that much each if p has the smaller sum, else none,
    # and the new token's number points into the middle of them. A border is right to 1e-9 of the sum of p + q = 2, so
    # to 2e-9 / S here where p and q are this close throughout: the number has to be further away from every border.
    B, V, n = 4096, 1100, 2
    g = np.random.default_rng(90)
    x = (np.round(g.standard_normal((B, V)) * 2048) / 1024 - 6.0).astype(np.float32)
    x[:, :512] -= 30.0             # (what the rows' sums are relative to: the sums are off by some 1e-7)
    x[:, 600:1024] -= 30.0
    x[:, V - 1] = np.log(0.02 * np.exp(x[:, :V - 2].astype(np.float64)).sum(1))
    x[:, V - 2], wanted = -7.0, 10.0 ** g.uniform(-8.5, -6, B)
    y = x + np.float32(5.25)       # (exactly so: the same distribution, of other numbers)
    y[:, V - 1] -= 1.0
    # q's sum above p's by `wanted` of it
    e = lambda z: np.exp(z.astype(np.float64))  # noqa: E731
    P = e(x).sum(1)
    y[:, V - 2] = np.log(e(x[:, V - 2]) + e(x[:, V - 1]) - e(y[:, V - 1] - 5.25) + wanted * P) + 5.25
    p, q = e(x) / P[:, None], e(y) / e(y).sum(1)[:, None]
    w = np.maximum(p - q, 0.0)
    c = np.cumsum(w, 1)
    # halfway to the last token, into the middle of the place of some token before it
    far = np.argsort(-w[:, :V - 1], 1)[np.arange(B), np.arange(B) % 5]
    far[(w[np.arange(B), far] == 0.0)] = V - 1
    u = ((c - 0.5 * w)[np.arange(B), far] / c[:, -1]).astype(np.float32)
    clear = 0.4 * w[np.arange(B), far] / c[:, -1] > 2e-9 / c[:, -1] + 2.0 ** -24 * u
    assert clear.sum() > B // 4 and (far[clear] != V - 1).sum() > B // 5
    rep = lambda z: torch.from_numpy(np.repeat(z, n, 0)).cuda()  # noqa: E731
    tokens, uniforms = np.full((B, n), V - 2), np.ones((B, n), np.float32)     # (the token of which q has more: turned away)
    uniforms[:, 0] = u
    got = tq.verify(rep(x), torch.from_numpy(tokens.ravel()).cuda(), torch.from_numpy(uniforms.ravel()).cuda(),
                    torch.arange(0, B * n + 1, n, device="cuda"), draft=rep(y),
                    parents=None if parents is None else torch.tensor(parents * B, device="cuda"))
    new = got.tokens.view(B, n)[:, 0].cpu().numpy()
    assert got.kept.tolist() == [1] * B
    wrong = (new != far) & clear
    assert not wrong.any(), (int(wrong.sum()), np.nonzero(wrong)[0][:5], wanted[wrong][:5])
