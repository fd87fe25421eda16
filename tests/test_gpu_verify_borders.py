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
