"""Rotary positions on fp32: sine and cosine, times the gain, are rounded to fp32 once, so with e = 2^-24 each
of the two products is off by e of itself for its factor and e for the product, and the sum by half a step:
2 e gain (|a| + |b|) + e |y|. (2.05: the angle in fp64, second order.)
"""

import numpy as np
import pytest
import torch

import rotation_lloyd_max_amd as tq
from oracle import attention as oat
from parity import as_f64

pytestmark = pytest.mark.gpu
E = 2.0 ** -24


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,heads,D,rot", [(1, 40, 128, 128), (700, 5, 64, 32), (33, 2, 256, 250), (1500, 3, 128, 64)])
def test_fp32_turns_are_off_by_the_roundings_alone(tokens, heads, D, rot, interleaved):
    g = np.random.default_rng([tokens, rot])
    x = torch.from_numpy(g.standard_normal((tokens, heads, D)).astype(np.float32)).cuda()
    pos = torch.from_numpy(g.integers(-(1 << 17), 1 << 17, tokens).astype(np.int32)).cuda()
    r = tq.rope_frequencies(rot, scaling="yarn", stretch=4.0, interleaved=interleaved)
    first, second = ((slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot)))
    a = np.abs(as_f64(x))
    for transposed in (False, True):
        got = as_f64(tq.rope(x, pos, r, transposed=transposed))
        ref = oat.rope(as_f64(x), pos.cpu().numpy(), r.inv_freq.cpu().numpy(), rot, interleaved, r.gain, transposed)
        bound = np.zeros_like(a)
        bound[..., first] = bound[..., second] = 2.05 * E * r.gain * (a[..., first] + a[..., second])
        bound[..., :rot] += 1.01 * E * np.abs(ref[..., :rot])
        err = np.abs(got - ref)
        assert np.all(err <= bound), float(np.max(err - bound))


@pytest.mark.parametrize("interleaved", [False, True])
def test_fp32_turns_are_off_by_four_roundings_in_the_mean(interleaved):
    # A rounding of a number of mantissa m is off by 2 e / sqrt(12) in the mean square, over m; over the
    # mantissas, 1 / m^2 has the mean 3 / (8 ln 2) = 0.541: 0.425 e of each number. Of an output these are the
    # two factors', one product's (the other stays in the fused sum) and the sum's: with half the square in
    # either product, 0.425 e sqrt(0.5 + 0.5 + 0.5 + 1) = 0.67 e of the norm. (8 % for the assumptions.)
    x = torch.randn((2000, 4, 128), generator=torch.Generator(device="cuda").manual_seed(4), device="cuda")
    pos = torch.arange(2000, device="cuda", dtype=torch.int32) * 61
    r = tq.rope_frequencies(128, interleaved=interleaved)
    got, ref = as_f64(tq.rope(x, pos, r)), oat.rope(as_f64(x), pos.cpu().numpy(), r.inv_freq.cpu().numpy(), 128, interleaved)
    assert np.linalg.norm(got - ref) <= 1.08 * 0.425 * 2.5 ** 0.5 * E * np.linalg.norm(ref)
