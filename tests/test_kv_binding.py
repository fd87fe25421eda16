"""Calls of the serving binding that must be refused, or must not be: gradients, overlapping outputs, index
values beyond 32 bits. CPU tensors, so that every check is shown to come before the library."""

import os

import numpy as np
import pytest
import torch

import rotation_lloyd_max_amd as tq

pytestmark = pytest.mark.skipif(not os.path.exists(tq.LIB_PATH), reason="libtq.so not built")
NOT_A_GPU = "must be on a GPU"      # the last check before the library: everything else was accepted


def cache(pages=2, heads=2, page=16, dim=64):
    halves = []
    for levels in (256, 8):
        rows = heads * page
        halves.append(tq.QWeight(torch.zeros((pages, rows, tq.words_per_row(dim, levels)), dtype=torch.int32),
                                 torch.zeros((pages, rows, dim // 32), dtype=torch.float16),
                                 torch.zeros(dim // 32, dtype=torch.int32), levels, 32, dim, rows, pages, 0))
    return tq.KVCache(halves[0], halves[1], heads, page)


def turn(x, **kw):
    return tq.rope(x, torch.zeros(x.shape[0], dtype=torch.int32), tq.Rope(torch.zeros(32, dtype=torch.float64), 64), **kw)


def attend(q, **kw):
    n = q.shape[0]
    return tq.kv_attend(cache(), q, torch.ones(n, dtype=torch.int32), torch.zeros((n, 1), dtype=torch.int32), **kw)


def test_gradients_are_not_lost_in_silence():
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16, requires_grad=True)
    for call in (lambda: turn(x), lambda: turn(x.detach(), out=torch.zeros_like(x, requires_grad=True)), lambda: attend(x),
                 lambda: attend(x * 2)):
        with pytest.raises(ValueError, match="gradient"):
            call()
    with torch.no_grad():
        for call in (lambda: turn(x), lambda: attend(x)):
            with pytest.raises(ValueError, match=NOT_A_GPU):
                call()
    with pytest.raises(ValueError, match=NOT_A_GPU):
        turn(x.detach())

    class Turn(torch.autograd.Function):       # the way to use them in training
        @staticmethod
        def forward(ctx, y):
            return turn(y)

    with pytest.raises(ValueError, match=NOT_A_GPU):
        Turn.apply(x)


def brute_force(x, y):
    def places(t):
        f = torch.arange(1 << 14)
        start = (t.data_ptr() - base.data_ptr()) // base.element_size()
        return set(f.as_strided(t.shape, t.stride(), start).flatten().tolist())
    base = x._base if x._base is not None else x
    return bool(places(x) & places(y))


def test_vectors_that_meet_are_found():
    # every pair of views of one buffer against the sets of their elements
    import itertools
    buf = torch.zeros(1 << 14)
    views = []
    for n, h, d in ((3, 2, 4), (1, 3, 8), (4, 1, 6)):
        group = []
        for ts, hs in ((32, 8), (8, 40), (16, 4), (6, 64), (100, 6), (d, n * d), (0, d)):
            for off in (0, 1, 3, 4, 8, 12, 20, 31, 64, 130):
                group.append(buf.as_strided((n, h, d), (ts, hs, 1), off))
        views.append(group)
    met = 0
    for group in views:
        for x, y in itertools.product(group, group):
            want = brute_force(x, y)
            met += want
            assert tq.kv._vectors_meet(x, y) == want, (x.shape, x.stride(), x.storage_offset(), y.stride(), y.storage_offset())
    assert 0 < met < sum(len(g) ** 2 for g in views)


def test_rope_outputs_that_overlap_the_input_in_part():
    wide = torch.zeros((5, 12, 64), dtype=torch.bfloat16)
    x = wide[1:3, 2:6]
    for bad in (wide[1:3, 3:7], wide[2:4, 2:6], wide[0:2, 4:8], wide.view(-1)[1 * 768 + 2 * 64 + 8:].as_strided((2, 4, 64), (768, 64, 1)),
                wide.as_strided((2, 4, 64), (64, 768, 1), 768 + 5 * 64)):
        with pytest.raises(ValueError, match="overlap"):
            turn(x, out=bad)
    for n, h in ((0, 4), (2, 0)):       # nothing to write: nothing to meet
        with pytest.raises(ValueError, match=NOT_A_GPU):
            turn(wide[1:1 + n, 2:2 + h], out=wide[1:1 + n, 3:3 + h])
    for good in (x, wide[1:3, 6:10], wide[3:5, 2:6], wide[1:3, 2:6].clone(), wide[0:1].view(-1)[:512].view(2, 4, 64)):
        with pytest.raises(ValueError, match=NOT_A_GPU):
            turn(x, out=good)


def test_load_outputs_that_overlap():
    c, slots = cache(), torch.zeros(3, dtype=torch.int64)
    buf = torch.zeros((6, 2, 64), dtype=torch.bfloat16)
    for k, v in ((buf[:3], buf[:3]), (buf[:3], buf[2:5])):
        with pytest.raises(ValueError, match="overlap"):
            tq.kv_load(c, slots, k_out=k, v_out=v)
    with pytest.raises(ValueError, match=NOT_A_GPU):
        tq.kv_load(c, slots, k_out=buf[:3], v_out=buf[3:])


def test_attention_outputs_that_overlap_the_queries_in_part():
    buf = torch.zeros((8, 4, 64), dtype=torch.bfloat16)
    wide = torch.zeros((3, 8, 64), dtype=torch.bfloat16)
    for q, out in ((buf[:3], buf[1:4]), (wide[:, :4], wide.view(-1)[:768].view(3, 4, 64)), (buf[:3], buf[:3].view(torch.float16))):
        with pytest.raises(ValueError, match="overlap"):
            attend(q, out=out)
    for q, out in ((buf[:3], buf[:3]), (buf[:3], buf[3:6])):
        with pytest.raises(ValueError, match=NOT_A_GPU):
            attend(q, out=out)


@pytest.mark.parametrize("dt", [torch.int64, torch.uint32, torch.uint64])
def test_index_values_beyond_their_type_stay_outside(dt):
    cpu = torch.device("cpu")
    values = [0, 5, 2 ** 31 - 1, 2 ** 31, 2 ** 32 - 1] + ([2 ** 32 + 3, 2 ** 40] if dt != torch.uint32 else []) + \
             ([-1, -2 ** 31 - 1, -2 ** 32 + 1] if dt == torch.int64 else []) + ([2 ** 64 - 1] if dt == torch.uint64 else [])
    t = torch.tensor(values, dtype=dt)
    got = tq.kv._as(t, torch.int32, cpu, "x", (len(values),))
    assert got.dtype == torch.int32 and got.tolist() == [max(-2 ** 31, min(2 ** 31 - 1, v)) for v in values]
    got = tq.kv._as(t, torch.int64, cpu, "x")
    assert got.dtype == torch.int64 and got.tolist() == [min(2 ** 63 - 1, v) for v in values]
    small = tq.kv._as(torch.tensor([-3, 7], dtype=torch.int16), torch.int32, cpu, "x")
    assert small.dtype == torch.int32 and small.tolist() == [-3, 7]


@pytest.mark.parametrize("rot,base,stretch,original", [(128, 1e4, 8.0, 4096), (64, 5e5, 32.0, 8192), (96, 1e4, 1.0, 2048), (6, 100.0, 3.5, 50)])
def test_frequencies_by_their_formulas(rot, base, stretch, original):
    i = np.arange(0, rot, 2)
    plain = base ** (-i / rot)
    turns = original * plain / (2 * np.pi)
    ramp = np.clip((turns - 1) / 31, 0, 1)          # linear in the turns
    want = {None: (plain, 1.0), "linear": (plain / stretch, 1.0),
            "ntk": ((base * stretch ** (rot / (rot - 2))) ** (-i / rot), 1.0),
            "yarn": (plain * ramp + plain / stretch * (1 - ramp), 0.1 * np.log(stretch) + 1)}
    for scaling, (f, gain) in want.items():
        r = tq.rope_frequencies(rot, base=base, scaling=scaling, stretch=stretch, original=original, device="cpu")
        np.testing.assert_allclose(r.inv_freq.numpy(), f, rtol=1e-13)
        assert abs(r.gain - gain) < 1e-15 and r.rot_dim == rot
