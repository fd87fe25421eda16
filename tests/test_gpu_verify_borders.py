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
    n = 0
    for b, x in enumerate(at):
        u = float(c["uniforms"][3 * b + 1])
        if abs(u * q[b, x] - p[b, x]) > 1e-12 * (u * q[b, x] + p[b, x]):
            n += 1
            assert first[b] == (u * q[b, x] < p[b, x]) == (path[3 * b + 1] == 1), (b, u, q[b, x], p[b, x])
    assert n > B * 0.99
