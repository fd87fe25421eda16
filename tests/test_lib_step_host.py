"""Host-side checks of include/tq_step.h and of the calls with several axes, without a GPU: exported
symbols, structs, and refusals with their status before any launch."""

import ctypes
import os
import re

import pytest
import torch

import rotation_lloyd_max_amd as tq
from rotation_lloyd_max_amd import kv, step
from test_lib_kv_host import BAD_CACHES, ERR_ALIGN, ERR_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, cache, rp

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "tq_step.h")

pytestmark = pytest.mark.skipif(not os.path.exists(tq.LIB_PATH), reason="libtq.so not built")


def header():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_exports_every_declared_symbol():
    names = sorted(set(re.findall(r"\b(tq_[a-z_]+)\s*\(", header())))
    handle = ctypes.CDLL(tq.LIB_PATH)
    for n in names:
        assert hasattr(handle, n), n
    assert sorted(s[0] for s in step.SIGNATURES) == names


def test_structs_match_the_header():
    body = re.findall(r"typedef struct \{([^}]*)\} (\w+);", header())
    fields = re.findall(r"\b(\w+)\s*[;,]", [b for b, n in body if n == "tq_kv_pool"][0])
    assert fields == [f[0] for f in step._KVPool._fields_]


# ---- refusals (fake pointers: nothing may be launched) ----------------------------------------

def pool(**kw):
    d = dict(free_pages=256, state=256, pages=4)
    d.update(kw)
    return step._KVPool(d["free_pages"], d["state"], d["pages"])


def plan(p=None, page=64, B=2, lens=256, counts=256, table=256, width=10, M=7, parents=None, shift=None, slots=256, pos=256,
         off=256, kvl=256, status=256, tree=None, words=0, left=None):
    return tq.lib().tq_kv_plan(p if p is not None else pool(), page, B, lens, counts, table, width, M, parents, shift, slots,
                               pos, off, kvl, status, tree, words, left, None)


def keep(p=None, c=None, page=64, B=2, lens=256, off=256, status=None, kept=256, path=None, M=7, table=256, width=10, out=256, left=None):
    return tq.lib().tq_kv_keep(p if p is not None else pool(), c, page, B, lens, off, status, kept, path, M, table, width, out,
                               left, None)


POOLS = [(dict(p=pool(pages=0)), ERR_ARG), (dict(p=pool(pages=(1 << 30) + 1)), ERR_ARG), (dict(p=pool(free_pages=None)), ERR_ARG),
         (dict(p=pool(state=None)), ERR_ARG), (dict(p=pool(state=258)), ERR_ALIGN), (dict(p=pool(free_pages=257)), ERR_ALIGN),
         (dict(page=0), ERR_ARG), (dict(page=65537), ERR_ARG), (dict(B=-1), ERR_ARG), (dict(B=65537), ERR_ARG),
         (dict(width=-1), ERR_ARG), (dict(width=1 << 25), ERR_ARG), (dict(lens=None), ERR_ARG), (dict(lens=258), ERR_ALIGN),
         (dict(table=None), ERR_ARG), (dict(table=1), ERR_ALIGN), (dict(left=2), ERR_ALIGN)]


@pytest.mark.parametrize("kw,status", POOLS)
def test_plan_and_keep_refuse_what_both_take(kw, status):
    assert plan(**kw) == keep(**kw) == status, tq.lib().tq_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), ERR_ARG), (dict(M=(1 << 24) + 1), ERR_ARG), (dict(counts=None), ERR_ARG), (dict(slots=None), ERR_ARG),
    (dict(slots=260), ERR_ALIGN), (dict(pos=None), ERR_ARG), (dict(off=None), ERR_ARG), (dict(kvl=None), ERR_ARG),
    (dict(status=None), ERR_ARG), (dict(tree=256), ERR_ARG), (dict(words=1), ERR_ARG), (dict(tree=256, words=65537), ERR_ARG),
    (dict(parents=3), ERR_ALIGN), (dict(shift=3), ERR_ALIGN), (dict(tree=258, words=1), ERR_ALIGN)])
def test_plan_refusals(kw, status):
    assert plan(**kw) == status, tq.lib().tq_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(kept=None), ERR_ARG), (dict(out=None), ERR_ARG), (dict(kept=258), ERR_ALIGN), (dict(off=258), ERR_ALIGN),
    (dict(status=258), ERR_ALIGN), (dict(out=258), ERR_ALIGN), (dict(path=256), ERR_ARG), (dict(path=256, c=cache(), page=32), ERR_ARG),
    (dict(path=256, c=cache(), p=pool(pages=5)), ERR_ARG), (dict(path=256, c=cache(), off=None), ERR_ARG),
    (dict(path=256, c=cache(), M=-1), ERR_ARG), (dict(path=256, c=cache(), M=(1 << 24) + 1), ERR_ARG),
    (dict(path=258, c=cache()), ERR_ALIGN)])
def test_keep_refusals(kw, status):
    assert keep(**kw) == status, tq.lib().tq_last_error()


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_moves_refuse_a_bad_cache(bad, status):
    assert keep(c=cache(**bad), path=256) == status, tq.lib().tq_last_error()


def test_null_pool_and_no_sequences():
    L = tq.lib()
    assert L.tq_kv_plan(None, 64, 2, 256, 256, 256, 10, 7, None, None, 256, 256, 256, 256, 256, None, 0, None, None) == ERR_ARG
    assert L.tq_kv_keep(None, None, 64, 2, 256, 256, None, 256, None, 0, 256, 10, 256, None, None) == ERR_ARG
    assert keep(B=0, lens=None, kept=None, out=None, table=None) == 0      # (nothing to launch)


def verify(t=256, tdt=tq.BF16, ts=100, d=256, ddt=tq.BF16, ds=100, flags=0, V=100, B=2, off=256, M=5, tok=256, par=None, u=256,
           temp=None, kept=256, out=256, path=256, ws=256, nbytes=1 << 40):
    return tq.lib().tq_verify(t, tdt, ts, d, ddt, ds, flags, V, B, off, M, tok, par, u, temp, kept, out, path, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(tdt=3), ERR_ARG), (dict(ddt=-1), ERR_ARG), (dict(flags=4), ERR_ARG), (dict(V=0), ERR_ARG), (dict(V=(1 << 28) + 1), ERR_ARG),
    (dict(B=-1), ERR_ARG), (dict(B=65537), ERR_ARG), (dict(M=-1), ERR_ARG), (dict(M=(1 << 24) + 1), ERR_ARG), (dict(t=None), ERR_ARG),
    (dict(off=None), ERR_ARG), (dict(tok=None), ERR_ARG), (dict(u=None), ERR_ARG), (dict(kept=None), ERR_ARG),
    (dict(out=None), ERR_ARG), (dict(path=None), ERR_ARG), (dict(t=257), ERR_ALIGN), (dict(d=257), ERR_ALIGN),
    (dict(t=258, tdt=tq.F32), ERR_ALIGN), (dict(tok=258), ERR_ALIGN), (dict(par=258), ERR_ALIGN), (dict(u=258), ERR_ALIGN),
    (dict(temp=258), ERR_ALIGN), (dict(ws=None), ERR_WORKSPACE), (dict(nbytes=16), ERR_WORKSPACE), (dict(ws=264), ERR_ALIGN)])
def test_verify_refusals(kw, status):
    assert verify(**kw) == status, tq.lib().tq_last_error()


def test_verify_of_no_sequences_and_its_workspace():
    assert verify(B=0, off=None, t=None, kept=None, M=0) == 0
    bad = ctypes.c_size_t(-1).value
    w = tq.lib().tq_verify_workspace
    for args in ((0, 1, 1, 0, 0), (1, -1, 1, 0, 0), (1, 1, -1, 0, 0), (1, 1, 1, 2, 0), (1, 1, 1, 0, 4)):
        assert w(*args) == bad
    assert w(131072, 64, 64 * 9, 1, 0) < 1 << 24      # (a small part of the logits)
    with pytest.raises(tq.TqError):
        tq.verify_workspace(0, 1, 1)


# ---- several axes ----------------------------------------------------------------------------

def rope(pos=256, stride=3, axes=3, axis=256, r=None, **kw):
    d = dict(x=256, dt=tq.BF16, tokens=3, heads=4, dim=128, xs=(512, 128), flags=0, out=4096, os_=(512, 128))
    d.update(kw)
    return tq.lib().tq_rope_axes(d["x"], d["dt"], d["tokens"], d["heads"], d["dim"], *d["xs"], pos, stride, axes, axis,
                                 r if r is not None else rp(), d["flags"], d["out"], *d["os_"], None)


def store(c, pos=256, stride=3, axes=3, axis=256, r=None, **kw):
    d = dict(k=256, v=256, dt=tq.BF16, tokens=3, slots=256)
    d.update(kw)
    return tq.lib().tq_kv_store_axes(c, d["k"], d["v"], d["dt"], d["tokens"], 1024, 128, 1024, 128, d["slots"],
                                     r if r is not None else rp(), pos, stride, axes, axis, None)


@pytest.mark.parametrize("kw,status", [
    (dict(axis=None), ERR_ARG), (dict(axes=0), ERR_ARG), (dict(axes=256), ERR_ARG), (dict(stride=-1), ERR_ARG),
    (dict(pos=None), ERR_ARG), (dict(pos=258), ERR_ALIGN), (dict(r=rp(rot_dim=130)), ERR_ARG), (dict(r=rp(inv_freq=260)), ERR_ALIGN),
    (dict(r=rp(interleaved=2)), ERR_ARG), (dict(dt=4), ERR_ARG), (dict(tokens=-1), ERR_ARG)])
def test_axes_refusals(kw, status):
    assert rope(**kw) == store(cache(), **kw) == status, tq.lib().tq_last_error()


def test_axes_of_no_tokens_and_of_a_bad_cache():
    assert rope(tokens=0, x=None, out=None) == 0 and store(cache(), tokens=0, k=None, v=None) == 0
    assert rope(dim=127) == ERR_UNSUPPORTED and rope(flags=2) == ERR_ARG and rope(out=256, os_=(1024, 128)) == ERR_ARG
    for bad, status in BAD_CACHES:
        assert store(cache(**bad)) == status
    assert tq.lib().tq_kv_store_axes(cache(), 256, 256, tq.BF16, 3, 1024, 128, 1024, 128, 256, None, 256, 3, 3, 256, None) == ERR_ARG


def test_which_pairs_and_frequencies_rope_axes_gives():
    r = tq.rope_axes((2, 1, 3), device="cpu")
    assert r.axis.tolist() == [0, 0, 1, 2, 2, 2] and r.rot_dim == 12
    assert torch.equal(r.inv_freq, tq.rope_frequencies(12, device="cpu").inv_freq)
    r = tq.rope_axes((2, 1, 3), order="cycle", scaling="yarn", stretch=8.0, device="cpu", interleaved=True)
    assert r.axis.tolist() == [0, 1, 2, 0, 2, 2] and r.interleaved
    y = tq.rope_frequencies(12, scaling="yarn", stretch=8.0, device="cpu")
    assert torch.equal(r.inv_freq, y.inv_freq) and r.gain == y.gain
    r = tq.rope_axes((2, 0, 3), restart=True, base=100.0, device="cpu")
    own = [tq.rope_frequencies(n, base=100.0, device="cpu").inv_freq for n in (4, 6)]
    assert torch.equal(r.inv_freq, torch.cat(own)) and r.axis.tolist() == [0, 0, 2, 2, 2]
    r = tq.rope_axes((2, 3), restart=True, order="cycle", base=100.0, device="cpu")
    assert r.axis.tolist() == [0, 1, 0, 1, 1]
    assert torch.equal(r.inv_freq, torch.stack([own[0][0], own[1][0], own[0][1], own[1][1], own[1][2]]))
    for bad in (dict(sections=()), dict(sections=(0, 0)), dict(sections=(3, -1)), dict(sections=[1] * 256),
                dict(sections=(1, 2), order="other"), dict(sections=(1,), scaling="other")):
        with pytest.raises(ValueError):
            tq.rope_axes(device="cpu", **bad)
    with pytest.raises(tq.TqError):
        tq.rope_axes((300, 300), device="cpu")


# ---- the binding's own checks (CPU tensors: every call must refuse before the library) -----------

NOT_A_GPU = "must be on a GPU"


def test_axes_binding():
    r = tq.rope_axes((16, 8, 8), device="cpu")
    x, pos = torch.zeros((5, 2, 64)), torch.zeros((3, 5), dtype=torch.int32)
    for p in (pos, pos[:1].expand(3, -1), pos.long(), pos.t().contiguous().t()):
        with pytest.raises(ValueError, match=NOT_A_GPU):
            tq.rope(x, p, r)
    for bad in (pos[0], pos[:, :4], pos[None]):
        with pytest.raises(ValueError, match="positions must be"):
            tq.rope(x, bad, r)
    with pytest.raises(TypeError):
        tq.rope(x, pos.float(), r)
    for axis in (r.axis[:31], r.axis.int(), torch.zeros(64, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="axis must be"):
            tq.rope(x, pos, tq.Rope(r.inv_freq, 64, axis=axis))
    with pytest.raises(ValueError, match="gradient"):
        tq.rope(x.requires_grad_(), pos, r)


def test_step_binding():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        tq.KVPool(i32(4).long(), i32(2))
    with pytest.raises(ValueError):
        tq.KVPool(i32(4), i32(3))
    pool = tq.kv_pool(4, device="cpu")
    assert pool.free.tolist() == [3, 2, 1, 0] and pool.state.tolist() == [4, 0]
    ok = dict(pool=pool, lens=i32(2), counts=i32(2), page_table=i32(2, 3), rows=5, page_tokens=16)
    for more in ({}, dict(parents=i32(5).long(), tree_words=1, shift=i32(2), left=i32(1)), dict(rows=0, tree_words=2)):
        with pytest.raises(ValueError, match=NOT_A_GPU):
            tq.kv_plan(**{**ok, **more})
    for bad in (dict(counts=i32(3)), dict(page_table=i32(2)), dict(page_table=i32(3, 2)), dict(page_table=i32(2, 3).long()),
                dict(page_table=i32(2, 6)[:, ::2]), dict(parents=i32(4)), dict(shift=i32(3)), dict(left=i32(2)), dict(left=i32(1).long()),
                dict(rows=-1), dict(tree_words=-1)):
        with pytest.raises(ValueError) as e:
            tq.kv_plan(**{**ok, **bad})
        assert NOT_A_GPU not in str(e.value)
    with pytest.raises(TypeError):
        tq.kv_plan(**{**ok, "lens": torch.zeros(2)})
    ok = dict(pool=pool, lens=i32(2), kept=i32(2), page_table=i32(2, 3), page_tokens=16)
    for more in ({}, dict(out=ok["lens"]), dict(out=i32(2), left=i32(1)), dict(q_offsets=i32(3), status=i32(2))):
        with pytest.raises(ValueError, match=NOT_A_GPU):
            tq.kv_keep(**{**ok, **more})
    both = i32(3)
    for bad in (dict(kept=i32(3)), dict(q_offsets=i32(2)), dict(status=i32(3)), dict(path=i32(4)), dict(out=i32(3)),
                dict(out=i32(2).long()), dict(lens=both[:2], out=both[1:])):
        with pytest.raises(ValueError) as e:
            tq.kv_keep(**{**ok, **bad})
        assert NOT_A_GPU not in str(e.value)
    # (lens of 64 bits are converted: their memory is not where the call may write)
    long = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError) as e:
        tq.kv_keep(**{**ok, "lens": long, "out": long.view(torch.int32)[:2]})
    assert NOT_A_GPU not in str(e.value)


def test_verify_binding():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    ok = dict(target=torch.zeros((5, 9)), tokens=i32(5), uniforms=torch.zeros(5), offsets=i32(3))
    for more in ({}, dict(draft=torch.zeros((5, 9), dtype=torch.float16), parents=i32(5).long(), temperature=torch.zeros(2)),
                 dict(target=torch.zeros((5, 20))[:, 3:12], target_kind="probabilities")):
        with pytest.raises(ValueError, match=NOT_A_GPU):
            tq.verify(**{**ok, **more})
    for bad in (dict(target=torch.zeros(9)), dict(target=torch.zeros((5, 18))[:, ::2]), dict(tokens=i32(4)), dict(uniforms=torch.zeros(4)),
                dict(uniforms=torch.zeros(5).double()), dict(offsets=i32(0)), dict(draft=torch.zeros((5, 8))),
                dict(draft=torch.zeros((4, 9))), dict(parents=i32(4)), dict(temperature=torch.zeros(3)),
                dict(temperature=torch.zeros(2).half()), dict(target_kind="other"), dict(ws=torch.zeros(1))):
        with pytest.raises(ValueError) as e:
            tq.verify(**{**ok, **bad})
        assert NOT_A_GPU not in str(e.value)
    with pytest.raises(TypeError):
        tq.verify(**{**ok, "target": torch.zeros((5, 9), dtype=torch.int32)})
    with pytest.raises(TypeError):
        tq.verify(**{**ok, "tokens": torch.zeros(5)})
