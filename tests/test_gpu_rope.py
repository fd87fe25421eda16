"""Rotary positions on the GPU against the oracle.

Bound, derived from the kernel's arithmetic in units e = 2^-24 (half a step of fp32): the angle
is exact to fp64, its fp32 form in half turns is off by at most e (an angle error of pi e), sine
and cosine by at most 4 e of 1 more (2 ulp), the gain's product by 2 e, each product and the sum
by e: together under 12 e gain (|a| + |b|) per element, then one rounding to the type.
"""

import numpy as np
import pytest
import torch

import rotation_lloyd_max_amd as tq
from oracle import attention as oat
from parity import as_f64

pytestmark = pytest.mark.gpu
DTS = [torch.float32, torch.bfloat16, torch.float16]
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def make(tokens, heads, D, dt, seed=0, far=1 << 18):
    g = np.random.default_rng([tokens, heads, D, seed])
    x = torch.from_numpy(g.standard_normal((tokens, heads, D)).astype(np.float32)).cuda().to(dt)
    pos = torch.from_numpy(g.integers(-far, far, tokens).astype(np.int32)).cuda()
    return x, pos


def check(got, x, pos, r, transposed=False):
    ref = oat.rope(as_f64(x), pos.cpu().numpy(), r.inv_freq.cpu().numpy(), r.rot_dim, r.interleaved, r.gain, transposed)
    a = np.abs(as_f64(x))
    room = np.zeros_like(a)
    h = r.rot_dim // 2
    i, j = (slice(0, r.rot_dim, 2), slice(1, r.rot_dim, 2)) if r.interleaved else (slice(0, h), slice(h, r.rot_dim))
    room[..., i] = room[..., j] = 12 * 2.0 ** -24 * r.gain * (a[..., i] + a[..., j])
    tiny = 2.0 ** -25 if x.dtype == torch.float16 else 0.0   # half a step of fp16's subnormals
    bound = room + HALF_STEP[x.dtype] * (np.abs(ref) + room) + tiny
    bound[..., r.rot_dim:] = 0.0
    err = np.abs(as_f64(got) - ref)
    assert np.all(err <= bound), float(np.max(err - bound))


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,heads,D,rot", [
    (1, 1, 2, 2), (1, 40, 128, 128), (3, 5, 64, 32), (7, 3, 80, 20), (129, 2, 96, 96), (2, 1, 1024, 1024), (65, 7, 128, 6),
    (1500, 9, 256, 64), (5, 3, 66, 66)])
def test_matches_oracle(dt, interleaved, tokens, heads, D, rot):
    x, pos = make(tokens, heads, D, dt)
    r = tq.rope_frequencies(rot, scaling="yarn", stretch=4.0, interleaved=interleaved)
    for transposed in (False, True):
        got = tq.rope(x, pos, r, transposed=transposed)
        torch.cuda.synchronize()
        check(got, x, pos, r, transposed)


def test_zero_tokens_and_heads():
    r = tq.rope_frequencies(64)
    for shape in ((0, 4, 64), (4, 0, 64)):
        x = torch.empty(shape, device="cuda")
        pos = torch.zeros(shape[0], dtype=torch.int32, device="cuda")
        assert tq.rope(x, pos, r).shape == shape


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("interleaved", [False, True])
def test_slices_in_place_and_odd_alignment(dt, interleaved):
    # query and key heads turned where they lie in a fused projection's output: nothing else changes
    g, pos = make(33, 12, 64, dt, seed=1)
    r = tq.rope_frequencies(64, interleaved=interleaved)
    wide = g.clone()
    out = tq.rope(wide[:, :10], pos, r, out=wide[:, :10])
    torch.cuda.synchronize()
    assert out.data_ptr() == wide.data_ptr()
    check(wide[:, :10], g[:, :10], pos, r)
    assert torch.equal(wide[:, 10:], g[:, 10:])
    # part of each head in place: the elements behind it stay
    part = tq.Rope(r.inv_freq[:5].clone(), 10, interleaved)
    same = g.clone()
    tq.rope(same, pos, part, out=same)
    torch.cuda.synchronize()
    check(same, g, pos, part)
    # heads before tokens in memory, and a base that 16-byte accesses cannot use
    t = g.transpose(0, 1).contiguous().transpose(0, 1)
    flat = torch.zeros(g.numel() + 1, dtype=dt, device="cuda")
    odd = flat[1:].view(g.shape)
    odd.copy_(g)
    want = tq.rope(g, pos, r)
    torch.cuda.synchronize()
    assert torch.equal(tq.rope(t, pos, r), want) and torch.equal(tq.rope(odd, pos, r), want)


def test_far_positions_keep_their_precision():
    x = torch.ones((2, 1, 2), device="cuda")
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    r = tq.Rope(torch.tensor([1.0], dtype=torch.float64, device="cuda"), 2)
    got = tq.rope(x, pos, r)
    torch.cuda.synchronize()
    check(got, x, pos, r)


def test_gradient_through_differences():
    # <w, rope(x + d) - rope(x)> = <d, rope^T(w)>: the map is linear; both sides in fp32, each
    # element off by at most 12 2^-24 gain (|a| + |b|) + half a step (see above)
    x, pos = make(17, 3, 64, torch.float32, seed=2)
    w, _ = make(17, 3, 64, torch.float32, seed=3)
    r = tq.rope_frequencies(48, interleaved=True, scaling="yarn", stretch=8.0)
    back = as_f64(tq.rope(w, pos, r, transposed=True))
    base = as_f64(tq.rope(x, pos, r))
    for e in ((0, 0, 0), (5, 1, 17), (16, 2, 47), (9, 0, 63)):
        x2 = x.clone()
        x2[e] += 1.0
        d = as_f64(x2)[e] - as_f64(x)[e]
        diff = as_f64(tq.rope(x2, pos, r)) - base
        left, right = float(np.sum(diff * as_f64(w))), float(back[e] * d)
        room = 30 * 2.0 ** -24 * r.gain * float(np.sum(np.abs(as_f64(w))[e[0], e[1]])) * float(np.max(np.abs(as_f64(x2)[e[0], e[1]])))
        assert abs(left - right) <= room, (e, left, right, room)


def test_another_stream():
    x, pos = make(64, 8, 128, torch.bfloat16, seed=5)
    r = tq.rope_frequencies(128)
    want = tq.rope(x, pos, r)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        got = tq.rope(x, pos, r)
    st.synchronize()
    assert torch.equal(got, want)
