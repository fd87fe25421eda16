"""The paged cache's write and read-back on the GPU: kv_store against the oracle's encode (and
byte for byte against tq.encode of the same rows), kv_load against the oracle's dequantize
and un-rotate, slots that are skipped, repeated or far beyond 32 bits, and what stays untouched."""

import numpy as np
import pytest
import torch

import rotation_lloyd_max_amd as tq
import workloads as wl
from oracle import attention as oat
from oracle import encode as oenc
from parity import as_f64, check_codes, check_scales, torch_to_np

pytestmark = pytest.mark.gpu
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}  # half the last subnormal step


def rows_of(tokens, heads, D, dt, seed):
    x = wl.kv_rows(wl.rng(991, D, seed), tokens, heads, D).reshape(tokens, heads, D)
    return torch.from_numpy(x).cuda().to(dt)


def picked(half, heads, page, slots):
    """The stored codes and scales of `slots`, [tokens * heads] rows."""
    s = np.asarray(slots)
    codes = torch_to_np(half.codes).reshape(half.E, heads, page, -1)[s // page, :, s % page]
    scales = torch_to_np(half.scales).reshape(half.E, heads, page, -1)[s // page, :, s % page]
    return codes.reshape(len(s) * heads, -1), scales.reshape(len(s) * heads, -1)


def slots_for(tokens, pages, page, seed):
    return np.random.default_rng(seed).permutation(pages * page)[:tokens].astype(np.int64)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 128)])
@pytest.mark.parametrize("kl,vl,heads,tokens,page", [(256, 8, 3, 37, 16), (16, 4, 8, 5, 64), (4, 16, 1, 1, 32), (8, 256, 20, 9, 48)])
def test_store_is_encode(dt, D, group, kl, vl, heads, tokens, page):
    pages = 4
    c = tq.kv_cache(pages, heads, D, page, kl, vl, group, group, k_seed=3, v_seed=8)
    k, v = rows_of(tokens, heads, D, dt, 1), rows_of(tokens, heads, D, dt, 2)
    slots = slots_for(tokens, pages, page, D + tokens)
    tq.kv_store(c, k, v, torch.from_numpy(slots).cuda())
    torch.cuda.synchronize()
    for half, x, seed in ((c.k, k, 3), (c.v, v, 8)):
        codes, scales = picked(half, heads, page, slots)
        flat = x.reshape(tokens * heads, D)
        qw = tq.encode(flat, half.levels, group, seed)
        torch.cuda.synchronize()
        np.testing.assert_array_equal(codes, torch_to_np(qw.codes)[0])
        np.testing.assert_array_equal(scales, torch_to_np(qw.scales)[0])
        ref = oenc.encode(as_f64(flat), half.levels, group, seed)
        check_codes(codes, ref, half.levels, D, f"{half.levels} levels")
        check_scales(scales, ref)
        # every other row of the cache is still zero
        mark = np.ones((pages, heads, page), dtype=bool)
        mark[slots // page, :, slots % page] = False
        assert not torch_to_np(half.codes).reshape(pages, heads, page, -1)[mark].any()
        assert not torch_to_np(half.scales).reshape(pages, heads, page, -1)[mark].any()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 128), (128, 32), (128, 20), (256, 128), (256, 2)])
def test_store_turns_the_keys(dt, interleaved, D, rot):
    heads, tokens, page, pages = 2, 21, 16, 3
    c = tq.kv_cache(pages, heads, D, page, 256, 16, 64, 64, k_seed=1, v_seed=2)
    k, v = rows_of(tokens, heads, D, dt, 3), rows_of(tokens, heads, D, dt, 4)
    slots = slots_for(tokens, pages, page, rot)
    pos = np.random.default_rng(rot).integers(0, 1 << 20, tokens).astype(np.int32)
    r = tq.rope_frequencies(rot, scaling="yarn", stretch=8.0, interleaved=interleaved)
    tq.kv_store(c, k, v, torch.from_numpy(slots).cuda(), rope=r, positions=torch.from_numpy(pos).cuda())
    torch.cuda.synchronize()
    turned = oat.rope(as_f64(k), pos, r.inv_freq.cpu().numpy(), rot, interleaved, r.gain)
    for half, x in ((c.k, turned), (c.v, as_f64(v))):
        codes, scales = picked(half, heads, page, slots)
        ref = oenc.encode(x.reshape(-1, D), half.levels, 64, half.seed)
        check_codes(codes, ref, half.levels, D, "turned")
        check_scales(scales, ref)


def test_store_takes_slices_of_a_projection():
    # k and v as strided slices (and at an address that 16-byte loads cannot use): same bytes
    heads, D, tokens, page = 4, 128, 19, 16
    for dt in (torch.float32, torch.bfloat16):
        wide = rows_of(tokens, 3 * heads, D, dt, 5)
        k, v = wide[:, heads:2 * heads], wide[:, 2 * heads:]
        slots = torch.from_numpy(slots_for(tokens, 2, page, 1)).cuda()
        a, b, o = (tq.kv_cache(2, heads, D, page) for _ in range(3))
        tq.kv_store(a, k, v, slots)
        tq.kv_store(b, k.contiguous(), v.contiguous(), slots)
        flat = torch.empty(k.numel() + 1, dtype=dt, device="cuda")
        ko = flat[1:].view(k.shape)
        ko.copy_(k)
        tq.kv_store(o, ko, v.transpose(0, 1).contiguous().transpose(0, 1), slots)
        torch.cuda.synchronize()
        for other in (b, o):
            assert torch.equal(a.k.codes, other.k.codes) and torch.equal(a.v.codes, other.v.codes)
            assert torch.equal(a.k.scales, other.k.scales) and torch.equal(a.v.scales, other.v.scales)


def test_store_skips_slots_outside_and_overwrites():
    heads, D, page, pages = 2, 64, 16, 2
    c = tq.kv_cache(pages, heads, D, page)
    x = rows_of(6, heads, D, torch.bfloat16, 6)
    first = torch.tensor([0, 1, 2, 3, 4, 5], device="cuda")
    tq.kv_store(c, x, x, first)
    before = (c.k.codes.clone(), c.v.codes.clone(), c.k.scales.clone(), c.v.scales.clone())
    bad = torch.tensor([-1, pages * page, -2 ** 63, 2 ** 62, 2 ** 32, -2 ** 32], device="cuda")
    tq.kv_store(c, -x, -x, bad)
    torch.cuda.synchronize()
    for a, b in zip(before, (c.k.codes, c.v.codes, c.k.scales, c.v.scales)):
        assert torch.equal(a, b)
    tq.kv_store(c, -x, -x, torch.tensor([-1, 1, -1, -1, 31, -1], device="cuda"))
    k, _ = tq.kv_load(c, torch.tensor([0, 1, 31], device="cuda"), out_dtype=torch.float32)
    k0, _ = tq.kv_load(c, first, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert torch.equal(k[0], k0[0]) and torch.equal(k[1], k0[1]) and not torch.equal(k[1], k[0])
    q = tq.kv_cache(pages, heads, D, page)
    tq.kv_store(q, -x[1:2], -x[1:2], torch.tensor([1], device="cuda"))
    assert torch.equal(tq.kv_load(q, torch.tensor([1], device="cuda"), out_dtype=torch.float32)[0], k[1:2])


def test_zero_nan_and_infinite_rows():
    heads, D, page = 1, 64, 16
    for levels in (256, 8):
        c = tq.kv_cache(1, heads, D, page, levels, levels, 32, 32)
        x = torch.zeros((5, 1, D), device="cuda")
        x[1] = float("nan")
        x[2, 0, 3] = float("inf")
        x[3] = 1e30          # group RMS beyond fp16: the scale saturates
        x[4] = 1e-30         # and below its smallest step
        tq.kv_store(c, x, x, torch.arange(5, device="cuda"))
        qw = tq.encode(x.view(5, D), levels, 32, 0)
        torch.cuda.synchronize()
        codes, scales = picked(c.k, 1, page, np.arange(5))
        want_c, want_s = torch_to_np(qw.codes)[0], torch_to_np(qw.scales)[0]
        np.testing.assert_array_equal(scales, want_s)
        np.testing.assert_array_equal(codes[[0, 3, 4]], want_c[[0, 3, 4]])
        k, _ = tq.kv_load(c, torch.arange(5, device="cuda"), out_dtype=torch.float32)
        assert not k[0].any() and torch.isnan(k[1]).all()


def load_bound(codes, scales, levels, group, D, ref, odt):
    # fp32 products and log2(D) butterfly stages: (log2 D + 3) 2^-24 ||w'_hat||_1 / sqrt(D) per
    # row, then one rounding to the output type
    w = oenc.dequant(codes, scales, levels, group, D)
    row = (int(np.log2(D)) + 3) * 2.0 ** -24 * np.sum(np.abs(w), axis=1, keepdims=True) / np.sqrt(D)
    return row + HALF_STEP[odt] * (np.abs(ref) + row) + TINY[odt]


@pytest.mark.parametrize("odt", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D,group", [(64, 32), (128, 64), (128, 128), (256, 32)])
@pytest.mark.parametrize("kl,vl,heads,tokens,page", [(256, 8, 3, 37, 16), (16, 4, 8, 5, 64), (4, 256, 1, 1, 32), (8, 16, 20, 301, 48)])
def test_load_matches_oracle(odt, D, group, kl, vl, heads, tokens, page):
    pages = max(2, -(-tokens // page) + 1)
    c = tq.kv_cache(pages, heads, D, page, kl, vl, group, group, k_seed=5, v_seed=6)
    k, v = rows_of(tokens, heads, D, torch.bfloat16, 7), rows_of(tokens, heads, D, torch.bfloat16, 8)
    slots = slots_for(tokens, pages, page, D)
    ts = torch.from_numpy(slots).cuda()
    tq.kv_store(c, k, v, ts)
    got = tq.kv_load(c, ts, out_dtype=odt)
    torch.cuda.synchronize()
    for half, g in ((c.k, got[0]), (c.v, got[1])):
        codes, scales = picked(half, heads, page, slots)
        ref = oenc.kv_fetch(codes, scales, half.levels, group, D, half.seed)
        err = np.abs(as_f64(g).reshape(-1, D) - ref)
        bound = load_bound(codes, scales, half.levels, group, D, ref, odt)
        assert np.all(err <= bound), float(np.max(err / bound))
    one = tq.kv_load(c, ts, out_dtype=odt, keys=False)
    assert one[0] is None and torch.equal(one[1], got[1])
    two = tq.kv_load(c, ts, out_dtype=odt, values=False)
    assert two[1] is None and torch.equal(two[0], got[0])


def test_load_agrees_with_fetch_and_repeats():
    heads, D, page, pages = 2, 128, 32, 3
    c = tq.kv_cache(pages, heads, D, page)
    x = rows_of(pages * page, heads, D, torch.bfloat16, 9)
    every = torch.arange(pages * page, device="cuda")
    tq.kv_store(c, x, x, every)
    for half, got in zip((c.k, c.v), tq.kv_load(c, every, out_dtype=torch.bfloat16)):
        whole = tq.kv_fetch(half, out_dtype=torch.bfloat16).view(pages, heads, page, D)
        torch.cuda.synchronize()
        a, b = as_f64(got.view(pages, page, heads, D).transpose(1, 2)), as_f64(whole)
        # two fp32 orders of the same sum, each rounded once: at most a step of bf16 apart
        assert np.all(np.abs(a - b) <= 2.0 ** -7 * np.maximum(np.abs(a), np.abs(b)) + 2.0 ** -18 * np.abs(b).max())
    again = torch.tensor([5, 5, 0, 5, -1, pages * page, 2 ** 40], device="cuda")
    k, v = tq.kv_load(c, again)
    torch.cuda.synchronize()
    full = tq.kv_load(c, every)[0]
    for i, s in enumerate((5, 5, 0, 5)):
        assert torch.equal(k[i], full[s])
    assert torch.isnan(k[4:]).all() and torch.isnan(v[4:]).all()


def test_slots_beyond_32_bits_of_bytes():
    # rows past 4 GiB of codes: 700000 pages of 48 tokens x 1 head x 256 bytes
    heads, D, page, pages = 1, 256, 48, 400000
    c = tq.kv_cache(pages, heads, D, page, 256, 4, 128, 128)
    assert c.k.codes.numel() * 4 > 1 << 32
    x = rows_of(4, heads, D, torch.bfloat16, 10)
    slots = torch.tensor([0, pages * page - 1, pages * page // 2, (1 << 32) // 256 + 7], device="cuda")
    tq.kv_store(c, x, x, slots)
    k, v = tq.kv_load(c, slots, out_dtype=torch.float32)
    small = tq.kv_cache(1, heads, D, 16, 256, 4, 128, 128)
    tq.kv_store(small, x, x, torch.arange(4, device="cuda"))
    ks, vs = tq.kv_load(small, torch.arange(4, device="cuda"), out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert torch.equal(k, ks) and torch.equal(v, vs)


def test_empty_calls():
    c = tq.kv_cache(1, 2, 64, 16)
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    x = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    tq.kv_store(c, x, x, none)
    k, v = tq.kv_load(c, none)
    assert k.shape == v.shape == (0, 2, 64)
