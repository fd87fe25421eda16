"""Rotary positions of several axes on the GPU against the oracle, pair by pair; bounds as derived in
test_gpu_rope.py (12 2^-24 gain (|a| + |b|) and one rounding); fp32 vectors are turned in fp64: one rounding
and 2^-31 gain (|a| + |b|) (the angle of position 2^18 in fp64: two roundings of its turns, 2 2^-53 2^18, times 2 pi: 2^-31).
One axis gives tq_rope's bits in the 16-bit types."""

import numpy as np
import pytest
import torch

import rotation_lloyd_max_amd as tq
from oracle import attention as oat
from parity import as_f64
from test_gpu_rope import DTS, HALF_STEP

pytestmark = pytest.mark.gpu


def reference(x, pos, r, transposed=False):
    """[T, heads, D] fp64: each axis turned alone by the oracle, the pairs of it taken."""
    axis, pos = r.axis.cpu().numpy(), pos.cpu().numpy()
    f, h = r.inv_freq.cpu().numpy(), r.rot_dim // 2
    out = np.array(as_f64(x))
    out[..., :r.rot_dim] *= r.gain
    for a in range(len(pos)):
        full = oat.rope(as_f64(x), pos[a], f, r.rot_dim, r.interleaved, r.gain, transposed)
        for i in np.nonzero(axis == a)[0]:
            for d in ((2 * i, 2 * i + 1) if r.interleaved else (i, i + h)):
                out[..., d] = full[..., d]
    return out


def check(got, x, pos, r, transposed=False):
    ref, a, h = reference(x, pos, r, transposed), np.abs(as_f64(x)), r.rot_dim // 2
    i, j = (slice(0, r.rot_dim, 2), slice(1, r.rot_dim, 2)) if r.interleaved else (slice(0, h), slice(h, r.rot_dim))
    room = np.zeros_like(a)
    near = pos.numel() == 0 or int(pos.abs().max()) <= 1 << 18
    room[..., i] = room[..., j] = (2.0 ** -31 if x.dtype == torch.float32 and near else 12 * 2.0 ** -24) * r.gain * (a[..., i] + a[..., j])
    tiny = 2.0 ** -25 if x.dtype == torch.float16 else 0.0
    bound = room + HALF_STEP[x.dtype] * (np.abs(ref) + room) + tiny
    bound[..., r.rot_dim:] = 0.0
    err = np.abs(as_f64(got) - ref)
    assert np.all(err <= bound), float(np.max(err - bound))


def make(tokens, heads, D, axes, dt, seed=0, far=1 << 18):
    g = np.random.default_rng([tokens, heads, D, axes, seed])
    x = torch.from_numpy(g.standard_normal((tokens, heads, D)).astype(np.float32)).cuda().to(dt)
    return x, torch.from_numpy(g.integers(-far, far, (axes, tokens)).astype(np.int32)).cuda()


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,heads,D,sections,kw", [
    (1, 1, 2, (1,), {}), (1, 40, 128, (16, 24, 24), {}), (3, 5, 64, (5, 0, 11), dict(order="cycle")),
    (7, 3, 80, (20, 20), dict(restart=True)), (129, 2, 96, (1, 2, 3, 4, 5), dict(order="cycle", restart=True)),
    (1500, 9, 256, (11, 30, 23), dict(scaling="yarn", stretch=4.0)), (65, 7, 128, (0, 3), dict(scaling="ntk", stretch=2.0)),
    (2, 1, 1024, (200, 312), {})])
def test_matches_oracle(dt, interleaved, tokens, heads, D, sections, kw):
    r = tq.rope_axes(sections, interleaved=interleaved, **kw)
    x, pos = make(tokens, heads, D, len(sections), dt)
    for transposed in (False, True):
        got = tq.rope(x, pos, r, transposed=transposed)
        torch.cuda.synchronize()
        check(got, x, pos, r, transposed)


@pytest.mark.parametrize("dt", DTS[1:])
def test_equal_axes_are_one_axis_bit_for_bit(dt):
    r = tq.rope_axes((16, 24, 24))
    x, pos = make(77, 6, 128, 1, dt, seed=1)
    want = tq.rope(x, pos[0], tq.rope_frequencies(128))
    for p in (pos.expand(3, -1), pos.repeat(3, 1), pos.repeat(3, 1).to(torch.int64)):
        assert torch.equal(tq.rope(x, p, r), want)
    one = tq.Rope(r.inv_freq, 128, axis=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    assert torch.equal(tq.rope(x, pos, one), want)


def test_strided_positions_slices_in_place_and_axes_beyond_the_positions():
    r = tq.rope_axes((8, 12, 12))
    g, pos = make(33, 12, 64, 3, torch.bfloat16, seed=2)
    wide = g.clone()
    padded = torch.full((3, 50), 7, dtype=torch.int32, device="cuda")
    padded[:, :33] = pos
    tq.rope(wide[:, :10], padded[:, :33], r, out=wide[:, :10])
    torch.cuda.synchronize()
    check(wide[:, :10], g[:, :10], pos, r)
    assert torch.equal(wide[:, 10:], g[:, 10:])
    check(tq.rope(g, pos.t().contiguous().t(), r), g, pos, r)      # tokens before axes in memory
    two = tq.rope(g, pos[:2], r)      # pairs of the third axis are not turned
    torch.cuda.synchronize()
    check(two, g, pos[:2], r)
    assert torch.equal(two[..., 20:32], g[..., 20:32]) and torch.equal(two[..., 52:64], g[..., 52:64])


def test_zero_tokens_far_positions_and_gradient():
    r = tq.rope_axes((16, 16))
    assert tq.rope(torch.empty((0, 4, 64), device="cuda"), torch.zeros((2, 0), dtype=torch.int32, device="cuda"), r).shape == (0, 4, 64)
    x, pos = make(2, 1, 64, 2, torch.float32, seed=3)
    pos = torch.tensor([[2 ** 31 - 1, -2 ** 31], [-2 ** 31, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    check(tq.rope(x, pos, r), x, pos, r)
    # the map is linear: <w, rope(x + d) - rope(x)> = <d, rope^T(w)>, room as in test_gpu_rope.py
    x, pos = make(17, 3, 64, 2, torch.float32, seed=4)
    w, _ = make(17, 3, 64, 2, torch.float32, seed=5)
    back, base = as_f64(tq.rope(w, pos, r, transposed=True)), as_f64(tq.rope(x, pos, r))
    for e in ((0, 0, 0), (5, 1, 17), (16, 2, 47), (9, 0, 63)):
        x2 = x.clone()
        x2[e] += 1.0
        d = as_f64(x2)[e] - as_f64(x)[e]
        left = float(np.sum((as_f64(tq.rope(x2, pos, r)) - base) * as_f64(w)))
        room = 30 * 2.0 ** -24 * float(np.sum(np.abs(as_f64(w))[e[0], e[1]])) * float(np.max(np.abs(as_f64(x2)[e[0], e[1]])))
        assert abs(left - float(back[e] * d)) <= room


@pytest.mark.parametrize("D,levels,rot,dt", [(128, (256, 8), (16, 24, 24), torch.bfloat16), (64, (16, 4), (8, 8), torch.float32),
                                             (256, (256, 16), (30, 30, 31), torch.float16)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_stored_keys_are_those_of_keys_turned_in_fp64(D, levels, rot, dt, interleaved):
    # equal axes: tq_kv_store's rows, byte for byte; axes of their own: each axis' rows where every
    # axis has the same position as it, which pins every pair
    r = tq.rope_axes(rot, interleaved=interleaved, order="cycle")
    n, heads, axes = 37, 3, len(rot)
    g = torch.Generator(device="cuda").manual_seed(7)
    k, v = (torch.randn((n, heads, D), generator=g, device="cuda").to(dt) for _ in range(2))
    pos = torch.randint(0, 9000, (axes, n), generator=g, device="cuda", dtype=torch.int32)
    slots = torch.randperm(96, generator=g, device="cuda")[:n]
    plain = tq.Rope(r.inv_freq, r.rot_dim, interleaved)

    def rows(rope, positions, keys=k):
        c = tq.kv_cache(3, heads, D, page_tokens=32, k_levels=levels[0], v_levels=levels[1])
        tq.kv_store(c, keys, v, slots, rope=rope, positions=positions)
        return c

    same, want = rows(r, pos[:1].expand(axes, n)), rows(plain, pos[0])
    for part in ("k", "v"):
        assert torch.equal(getattr(same, part).codes, getattr(want, part).codes)
        assert torch.equal(getattr(same, part).scales, getattr(want, part).scales)
    # keys with one axis' pairs only: the other pairs are zero and stay zero under any turn
    mixed_axes = r.axis.long()
    for a in range(axes):
        only = torch.zeros(D, dtype=torch.bool, device="cuda")
        i = torch.nonzero(mixed_axes == a).flatten()
        only[2 * i if interleaved else i] = True
        only[2 * i + 1 if interleaved else i + r.rot_dim // 2] = True
        part = torch.where(only, k, torch.zeros_like(k))
        got, want = rows(r, pos, part), rows(plain, pos[a], part)
        assert torch.equal(got.k.codes, want.k.codes) and torch.equal(got.k.scales, want.k.scales)


def test_captured_with_new_positions():
    r = tq.rope_axes((16, 24, 24))
    x, pos = make(5, 40, 128, 3, torch.bfloat16, seed=8)
    out = torch.empty_like(x)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        tq.rope(x, pos, r, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tq.rope(x, pos, r, out=out)
    for step in range(3):
        pos.add_(step)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, tq.rope(x, pos, r))
