"""Host-side checks of the entry points of include/tq_kv.h that need no GPU: exported symbols,
refusals with their status before any launch, and the rotary frequencies."""

import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import rotation_lloyd_max_amd as tq
from rotation_lloyd_max_amd import kv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "tq_kv.h")

pytestmark = pytest.mark.skipif(not os.path.exists(tq.LIB_PATH),
                                reason="libtq.so not built (run __graft_entry__.build())")

ERR_ARG, ERR_UNSUPPORTED, ERR_ALIGN, ERR_WORKSPACE = -1, -2, -3, -4


def test_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(tq_[a-z_]+)\s*\(", text)))
    handle = ctypes.CDLL(tq.LIB_PATH)
    for n in names:
        assert hasattr(handle, n), n
    assert sorted(s[0] for s in kv.SIGNATURES) == names


def test_structs_match_the_header():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    for name, cls in (("tq_kv_cache", kv._KVCache), ("tq_rope_params", kv._RopeParams)):
        body = re.findall(r"typedef struct \{([^}]*)\} (\w+);", text)
        fields = re.findall(r"\b(\w+)\s*[;,]", [b for b, n in body if n == name][0])
        assert fields == [f[0] for f in cls._fields_]


# ---- refusals (fake pointers: nothing may be launched) ---------------------------------------

def half(**kw):
    d = dict(codes=256, scales=256, signs=256, n_levels=256, group=64, K=128, N=8 * 64, E=4)
    d.update(kw)
    return tq._QWeight(d["codes"], d["scales"], d["signs"], d["n_levels"], d["group"], d["K"], d["N"], d["E"])


def cache(k=None, v=None, heads=8, page=64):
    return kv._KVCache(half(**(k or {})), half(n_levels=8, **(v or {})), heads, page)


def rp(**kw):
    d = dict(inv_freq=256, rot_dim=64, interleaved=0, gain=1.0)
    d.update(kw)
    return kv._RopeParams(d["inv_freq"], d["rot_dim"], d["interleaved"], d["gain"])


def store(c, k=256, v=256, dt=tq.BF16, tokens=3, strides=(1024, 128, 1024, 128), slots=256, r=None, pos=256):
    return tq.lib().tq_kv_store(c, k, v, dt, tokens, *strides, slots, r, pos, None)


def load(c, slots=256, tokens=3, k=256, v=256, dt=tq.BF16):
    return tq.lib().tq_kv_load(c, slots, tokens, k, v, dt, None)


def attend(c, q=256, qdt=tq.BF16, qh=32, stride=4096, B=2, off=256, M=4, lens=256, table=256, width=10, tree=None,
           words=0, scale=0.1, out=256, odt=tq.BF16, ws=256, nbytes=1 << 40):
    return tq.lib().tq_kv_attend(c, q, qdt, qh, stride, B, off, M, lens, table, width, tree, words, scale, out, odt,
                                 ws, nbytes, None)


BAD_CACHES = [
    (dict(k=dict(n_levels=3)), ERR_UNSUPPORTED), (dict(k=dict(n_levels=32)), ERR_UNSUPPORTED),
    (dict(k=dict(K=96), v=dict(K=96)), ERR_UNSUPPORTED), (dict(k=dict(K=512), v=dict(K=512)), ERR_UNSUPPORTED),
    (dict(k=dict(group=16)), ERR_UNSUPPORTED), (dict(v=dict(group=48)), ERR_UNSUPPORTED),
    (dict(k=dict(K=64, group=128), v=dict(K=64)), ERR_UNSUPPORTED),
    (dict(k=dict(N=511)), ERR_ARG), (dict(v=dict(E=5)), ERR_ARG), (dict(v=dict(K=64)), ERR_ARG),
    (dict(k=dict(E=0)), ERR_ARG), (dict(k=dict(E=1 << 31)), ERR_ARG), (dict(heads=0), ERR_ARG),
    (dict(page=0), ERR_ARG), (dict(page=24), ERR_ARG), (dict(page=1 << 17), ERR_ARG),
    (dict(k=dict(codes=None)), ERR_ARG), (dict(v=dict(scales=None)), ERR_ARG), (dict(k=dict(signs=None)), ERR_ARG),
    (dict(k=dict(codes=264)), ERR_ALIGN), (dict(v=dict(scales=258)), ERR_ALIGN), (dict(v=dict(signs=257)), ERR_ALIGN),
]


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_every_call_refuses_a_bad_cache(bad, status):
    c = cache(**bad)
    assert store(c) == load(c) == attend(c) == status, tq.lib().tq_last_error()
    assert tq.lib().tq_kv_attend_workspace(c, 32, 2, 4) == ctypes.c_size_t(-1).value


def test_null_cache():
    assert store(None) == load(None) == attend(None) == ERR_ARG


@pytest.mark.parametrize("kw,status", [
    (dict(dt=3), ERR_ARG), (dict(tokens=-1), ERR_ARG), (dict(tokens=(1 << 30) + 1), ERR_ARG), (dict(k=None), ERR_ARG),
    (dict(v=None), ERR_ARG), (dict(slots=None), ERR_ARG), (dict(k=257), ERR_ALIGN), (dict(slots=260), ERR_ALIGN),
    (dict(r=rp(rot_dim=130)), ERR_ARG), (dict(r=rp(rot_dim=7)), ERR_ARG), (dict(r=rp(rot_dim=0)), ERR_ARG),
    (dict(r=rp(inv_freq=None)), ERR_ARG), (dict(r=rp(inv_freq=260)), ERR_ALIGN), (dict(r=rp(interleaved=2)), ERR_ARG),
    (dict(r=rp(), pos=None), ERR_ARG), (dict(r=rp(), pos=258), ERR_ALIGN)])
def test_store_refusals(kw, status):
    assert store(cache(), **kw) == status, tq.lib().tq_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(dt=-1), ERR_ARG), (dict(tokens=-1), ERR_ARG), (dict(slots=None), ERR_ARG), (dict(slots=4), ERR_ALIGN),
    (dict(k=264), ERR_ALIGN), (dict(v=8), ERR_ALIGN)])
def test_load_refusals(kw, status):
    assert load(cache(), **kw) == status, tq.lib().tq_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(qdt=tq.F32), ERR_UNSUPPORTED), (dict(odt=tq.F32), ERR_UNSUPPORTED), (dict(qdt=9), ERR_UNSUPPORTED),
    (dict(qh=12), ERR_ARG), (dict(qh=0), ERR_ARG), (dict(B=-1), ERR_ARG), (dict(B=65537), ERR_ARG),
    (dict(M=-1), ERR_ARG), (dict(M=(1 << 24) + 1), ERR_ARG), (dict(off=None, M=5), ERR_ARG), (dict(width=-1), ERR_ARG),
    (dict(width=1 << 26), ERR_ARG), (dict(words=1), ERR_ARG), (dict(tree=256), ERR_ARG), (dict(scale=math.inf), ERR_ARG),
    (dict(scale=math.nan), ERR_ARG), (dict(q=None), ERR_ARG), (dict(out=None), ERR_ARG), (dict(lens=None), ERR_ARG),
    (dict(table=None), ERR_ARG), (dict(q=264), ERR_ALIGN), (dict(stride=4100), ERR_ALIGN), (dict(out=8), ERR_ALIGN),
    (dict(lens=2), ERR_ALIGN), (dict(table=2), ERR_ALIGN), (dict(off=2), ERR_ALIGN), (dict(tree=2, words=1), ERR_ALIGN),
    (dict(B=0, M=4, off=None), ERR_ARG), (dict(qh=1024, M=1 << 22, off=256), ERR_ARG),
    (dict(qh=64, M=1 << 18, off=256, width=1 << 24), ERR_ARG)])
def test_attend_refusals(kw, status):
    assert attend(cache(), **kw) == status, tq.lib().tq_last_error()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("qh,B,M", [(8, 1, 1), (32, 1, 1), (32, 64, 64), (32, 1, 16), (32, 1, 1 << 20), (1024, 65536, 1 << 20), (8, 0, 0)])
def test_attend_workspace_is_bounded(D, qh, B, M):
    n = tq.lib().tq_kv_attend_workspace(cache(dict(K=D, group=32), dict(K=D, group=32)), qh, B, M)
    assert n <= 69 * 10 ** 6 and (n > 0) == (M > 0)


def test_empty_calls_do_nothing():
    c = cache()
    assert store(c, tokens=0, k=None, v=None, slots=None) == 0
    assert load(c, tokens=0, slots=None) == 0 and load(c, k=None, v=None) == 0
    assert attend(c, M=0, q=None, out=None) == 0 and attend(c, B=0, M=0) == 0
    assert rope(x=None, tokens=0) == 0 and rope(heads=0) == 0


def rope(x=256, dt=tq.BF16, tokens=3, heads=4, dim=128, xs=(512, 128), pos=256, r=None, flags=0, out=4096, os_=(512, 128)):
    return tq.lib().tq_rope(x, dt, tokens, heads, dim, *xs, pos, r if r is not None else rp(), flags, out, *os_, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=4), ERR_ARG), (dict(dim=0), ERR_UNSUPPORTED), (dict(dim=127), ERR_UNSUPPORTED), (dict(dim=2048), ERR_UNSUPPORTED),
    (dict(tokens=-1), ERR_ARG), (dict(heads=-1), ERR_ARG), (dict(heads=65537), ERR_ARG), (dict(flags=2), ERR_ARG),
    (dict(x=None), ERR_ARG), (dict(out=None), ERR_ARG), (dict(x=257), ERR_ALIGN), (dict(out=4097), ERR_ALIGN),
    (dict(out=256, os_=(1024, 128)), ERR_ARG), (dict(os_=(0, 128)), ERR_ARG), (dict(os_=(512, 0)), ERR_ARG),
    (dict(pos=None), ERR_ARG), (dict(r=rp(rot_dim=130)), ERR_ARG), (dict(r=rp(inv_freq=None)), ERR_ARG)])
def test_rope_refusals(kw, status):
    assert rope(**kw) == status, tq.lib().tq_last_error()


# ---- frequencies -----------------------------------------------------------------------------

def test_frequencies():
    f = tq.rope_frequencies(128, base=1e6, device="cpu")
    np.testing.assert_allclose(f.inv_freq.numpy(), 1e6 ** (-np.arange(0, 128, 2) / 128), rtol=1e-14)
    assert f.gain == 1.0 and f.inv_freq.dtype == torch.float64
    lin = tq.rope_frequencies(128, base=1e6, scaling="linear", stretch=4.0, device="cpu")
    np.testing.assert_allclose(lin.inv_freq.numpy(), f.inv_freq.numpy() / 4.0, rtol=1e-14)
    # NTK: the slowest frequency is divided by the stretch, the fastest kept
    ntk = tq.rope_frequencies(128, base=1e6, scaling="ntk", stretch=8.0, device="cpu").inv_freq.numpy()
    np.testing.assert_allclose([ntk[0], ntk[-1]], [1.0, f.inv_freq.numpy()[-1] / 8.0], rtol=1e-12)
    # YARN: fewer than one turn in the original length divided, more than 32 kept, a ramp between
    y = tq.rope_frequencies(128, base=1e4, scaling="yarn", stretch=16.0, original=4096, device="cpu")
    p = tq.rope_frequencies(128, base=1e4, device="cpu").inv_freq.numpy()
    turns, ratio = 4096 * p / (2 * np.pi), y.inv_freq.numpy() / p
    np.testing.assert_allclose(ratio[turns > 32], 1.0, rtol=1e-14)
    np.testing.assert_allclose(ratio[turns < 1], 1 / 16, rtol=1e-14)
    assert np.all(np.diff(ratio) <= 1e-15) and abs(y.gain - (0.1 * math.log(16.0) + 1.0)) < 1e-15
    for s in (None, "linear", "ntk", "yarn"):
        same = tq.rope_frequencies(64, scaling=s, stretch=1.0, device="cpu")
        np.testing.assert_allclose(same.inv_freq.numpy(), 1e4 ** (-np.arange(0, 64, 2) / 64), rtol=1e-14)
        assert same.gain == 1.0


@pytest.mark.parametrize("kw", [dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=64, base=0.0), dict(rot_dim=64, base=math.inf),
                                dict(rot_dim=64, scaling="linear", stretch=0.5), dict(rot_dim=64, stretch=math.nan),
                                dict(rot_dim=64, scaling="yarn", original=0.0), dict(rot_dim=2, scaling="ntk", stretch=2.0),
                                dict(rot_dim=2048)])
def test_frequency_refusals(kw):
    with pytest.raises(tq.TqError):
        tq.rope_frequencies(device="cpu", **kw)
    with pytest.raises(ValueError):
        tq.rope_frequencies(64, scaling="other", device="cpu")


# ---- the binding's own checks (CPU tensors: every call must refuse before the library) ---------

def cpu_cache(pages=2, heads=2, page=16, dim=64, levels=(256, 8), group=32):
    halves = []
    for L in levels:
        rows = heads * page
        halves.append(tq.QWeight(torch.zeros((pages, rows, tq.words_per_row(dim, L)), dtype=torch.int32),
                                 torch.zeros((pages, rows, dim // group), dtype=torch.float16),
                                 torch.zeros(dim // 32, dtype=torch.int32), L, group, dim, rows, pages, 0))
    return tq.KVCache(halves[0], halves[1], heads, page)


def test_cache_checks_its_tensors():
    c = cpu_cache()
    for field, bad in (("codes", c.k.codes[:1]), ("codes", c.k.codes.float()), ("scales", c.k.scales[:, :, :1]),
                       ("scales", c.k.scales.float()), ("signs", c.k.signs[:1]), ("levels", 8), ("E", 3), ("levels", 3)):
        k = tq.QWeight(**{**c.k.__dict__, field: bad})
        with pytest.raises(ValueError):
            tq.KVCache(k, c.v, 2, 16)


def test_binding_refusals():
    c = cpu_cache()
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError):   # not on a GPU
        tq.kv_store(c, x, x, slots)
    for bad in (dict(k=x[:, :1]), dict(v=x.float()), dict(slots=slots[:2]), dict(k=x.transpose(1, 2)),
                dict(rope=tq.Rope(torch.zeros(32, dtype=torch.float64), 64)),
                dict(rope=tq.Rope(torch.zeros(32), 64), positions=slots),
                dict(rope=tq.Rope(torch.zeros(31, dtype=torch.float64), 64), positions=slots)):
        with pytest.raises(ValueError):
            tq.kv_store(c, **{**dict(k=x, v=x, slots=slots), **bad})
    with pytest.raises(TypeError):
        tq.kv_store(c, x, x, slots.float())
    with pytest.raises(ValueError):
        tq.kv_load(c, slots, out_dtype=torch.float16, k_out=torch.empty((3, 2, 64)))
    with pytest.raises(ValueError):
        tq.kv_load(c, slots, out_dtype=torch.float32, k_out=torch.empty((2, 2, 64)))
    q, lens, table = torch.zeros((3, 4, 64), dtype=torch.float16), torch.ones(3, dtype=torch.int32), torch.zeros((3, 2), dtype=torch.int32)
    for bad in (dict(q=q[:, :, :32]), dict(q=torch.zeros((3, 8, 64), dtype=torch.float16)[:, ::2]), dict(page_table=table[:2]),
                dict(page_table=table[0]), dict(q_offsets=lens), dict(tree=torch.zeros((2, 1), dtype=torch.int32)),
                dict(tree=torch.zeros((3, 1), dtype=torch.int64)), dict(out=torch.zeros((3, 4, 63), dtype=torch.float16)),
                dict(out=q.clone(), out_dtype=torch.bfloat16)):
        with pytest.raises(ValueError):
            tq.kv_attend(c, **{**dict(q=q, kv_lens=lens, page_table=table), **bad})
    with pytest.raises(tq.TqError):   # three query heads do not share two key heads
        tq.kv_attend(c, torch.zeros((3, 3, 64), dtype=torch.float16), lens, table)
    r = tq.Rope(torch.zeros(32, dtype=torch.float64), 64)
    for bad in (dict(positions=slots[:2]), dict(out=x.float()), dict(out=x[:1].expand(3, 2, 64)), dict(x=x[0])):
        with pytest.raises(ValueError):
            tq.rope(**{**dict(x=x, positions=slots, rope=r), **bad})
