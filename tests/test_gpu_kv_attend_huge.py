"""Attention with scores beyond 2^20, where a step of fp32 is a sizeable exponent: each query points at
one key that the cache holds twice, far from one another, so that these two share all the weight and the
output is the mean of their values, whatever the scores' size.

Bound: the weights are equal (the two scores are the same number) and the others' are 0, so what is left
of test_gpu_kv_attend's bound is the rounding of p and of the decoded values, 3 u + 2^-18 + n 2^-24 of
the mean of |v|, and out's half step.
"""

import numpy as np
import pytest
import torch

from oracle import hadamard as ohd
from parity import as_f64
from test_gpu_kv_attend import HALF_STEP, U, Batch, check, queries, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,share", [(1, 3), (5, 3), (40, 2), (150, 2)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_two_equal_scores_of_any_size(D, n, share):
    bt = Batch([320 + n], heads=1, D=D, page=48, kg=64, vg=64, kl=256, vl=256, seed=n)
    bt.cache.k.scales.fill_(1.0)
    codes = bt.cache.k.codes.view(-1, 48, bt.cache.k.codes.shape[-1])
    for j in range(160):                       # token j + 160 has the key of token j
        a, b = int(bt.slots[0][j]), int(bt.slots[0][j + 160])
        codes[b // 48, b % 48] = codes[a // 48, a % 48].clone()
    bt.refresh()
    kp, vp = bt.rows[0][0][:, 0], bt.rows[1][0][:, 0]
    which = (np.arange(n * share) * 37 % 160).reshape(n, share)
    keys = ohd.unrotate(kp[which.reshape(-1)], 21).reshape(n, share, D)
    for size in (3e6, 1e9, -1e13, 1e20):
        scale = D ** -0.5 if size > 0 else -D ** -0.5
        q = torch.from_numpy((keys * size).astype(np.float32)).cuda().to(torch.bfloat16)
        out = as_f64(run(bt, q, [n], scale=scale))
        qr = ohd.rotate(as_f64(q).reshape(-1, D), 21).reshape(n, share, D)
        for i in range(n):
            for h in range(share):
                j = which[i, h]
                s = scale * (kp[:320 + i + 1] @ qr[i, h])
                E = abs(scale) * (3 * U + (D + 16) * 2.0 ** -24 + 2.0 ** -19 * D ** 0.5) * np.abs(kp).sum(1).max() * np.abs(qr[i, h]).max()
                rest = np.delete(s, [j, j + 160])
                assert s[j] == s[j + 160] and rest.max() + 2 * E + 60 < s[j], (i, h)
                want = ohd.unrotate((vp[j] + vp[j + 160])[None] / 2, 22)[0]
                rel = 3 * U + 2.0 ** -18 + len(s) * 2.0 ** -24
                room = rel * np.linalg.norm(np.abs(vp[j]) + np.abs(vp[j + 160])) / 2 + HALF_STEP[torch.bfloat16] * np.linalg.norm(want) * 1.01
                err = np.linalg.norm(out[i, h] - want)
                assert err <= room, (size, i, h, err, room)
    q = queries(n, share, D, torch.bfloat16)
    check(run(bt, q, [n]), bt, q, [n], D ** -0.5, only=set(range(0, n, 11)))
