"""Attention over the packed cache where its own roundings are known, so that the bounds are tight
enough to show one token of thousands missing, counted twice or taken from another row.

The kernel decodes to fp16: a centroid rounded to fp16 times the row's scale, rounded to fp16 (scales
between 2^-4 and 2^13, as here, enter as they are). With these values as the oracle's, what is left of
each part is, per element and relative to the sum of |terms|:
  sums       n tokens (D elements of a score) in fp32, n 2^-23: a matrix instruction may cut where
             fp32 would round
  q = 0      all weights are the same number, so the output is the mean of the tokens it sees:
             nothing but the sums, 64 2^-24 for the normalisation, the join and the rotation back,
             and out's own half step (2^-25 where it is subnormal)
  integer q  R_k q has integers of at most 2^11 before its factor 1 / sqrt(D), exact in fp16: scores
             are off by E = |scale| (D + 16) 2^-23 sum |q'_d k'_d| + 2^-20 max |s|, weights by
             e^(2 E), half a step of fp16 and 2^-32 of the largest (fp16's subnormals: 2^-25 below a
             reference of 2^7).
"""

import numpy as np
import pytest
import torch

import rotation_lloyd_max_amd as tq
from oracle import attention as oat
from oracle import codebook as ocb
from oracle import encode as oenc
from oracle import hadamard as ohd
from parity import as_f64, torch_to_np
from test_gpu_kv_attend import Batch, run, tree_rows

pytestmark = pytest.mark.gpu
U = 2.0 ** -11


def decoded(bt):
    """The rows as the kernel holds them: per half and sequence [tokens, heads, D], in fp64."""
    halves = []
    for half in (bt.cache.k, bt.cache.v):
        codes = torch_to_np(half.codes).reshape(half.E, bt.heads, bt.page, -1)
        scales = torch_to_np(half.scales).reshape(half.E, bt.heads, bt.page, -1)
        c16 = ocb.centroids(half.levels).astype(np.float32).astype(np.float16)
        per = []
        for s in bt.slots:
            if len(s) == 0:
                per.append(np.zeros((0, bt.heads, bt.D)))
                continue
            cc = codes[s // bt.page, :, s % bt.page].reshape(len(s) * bt.heads, -1)
            ss = scales[s // bt.page, :, s % bt.page].reshape(len(s) * bt.heads, -1).view(np.float16)
            assert ss.min() >= 2.0 ** -4 and ss.max() < 2.0 ** 13
            w = c16[oenc.unpack(cc, half.levels, bt.D)] * np.repeat(ss, half.group, axis=-1)
            assert w.dtype == np.float16
            per.append(w.astype(np.float64).reshape(len(s), bt.heads, bt.D))
        halves.append(per)
    return halves


def masks(bt, counts, tree):
    m = 0
    for b, n in enumerate(counts):
        for i in range(n):
            yield m, b, oat.seen(bt.lens[b], n, i, None if tree is None else tree[m])
            m += 1


def check_means(bt, share, counts, tree=None, only=None, offsets=True):
    q = torch.zeros((sum(counts), bt.heads * share, bt.D), dtype=torch.bfloat16, device="cuda")
    out = as_f64(run(bt, q, counts if offsets else None, tree, out_dtype=torch.float16))
    _, v = decoded(bt)
    sums = [np.concatenate([np.zeros((1, bt.heads, bt.D)), np.cumsum(x, axis=0)]) for x in v]
    sizes = [np.concatenate([np.zeros((1, bt.heads, bt.D)), np.cumsum(np.abs(x), axis=0)]) for x in v]
    for m, b, mask in masks(bt, counts, tree):
        if only is not None and m not in only:
            continue
        n = int(mask.sum())
        if n == 0:
            assert not out[m].any()
            continue
        if mask[:n].all():
            mean, size = sums[b][n] / n, sizes[b][n] / n
        else:
            mean, size = v[b][mask].mean(axis=0), np.abs(v[b][mask]).mean(axis=0)
        want = ohd.unrotate(mean, 22)
        room = ((n * 2.0 ** -23 + 64 * 2.0 ** -24) * np.linalg.norm(size, axis=-1)
                + U * 1.01 * np.linalg.norm(want, axis=-1) + 2.0 ** -25 * bt.D ** 0.5)
        err = np.linalg.norm(out[m].reshape(bt.heads, share, bt.D) - want[:, None], axis=-1)
        assert (err <= room[:, None]).all(), (m, b, n, (err / room[:, None]).max())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kl,vl", [(256, 8), (16, 16), (4, 256), (256, 4), (8, 256), (16, 8)])
def test_means_of_every_format(D, kl, vl):
    lens = [1, 16, 17, 33, 100, 259, 2000]
    for kg, vg in ((32, 32), (64, 64), (128, 128)):
        bt = Batch(lens, heads=2, D=D, page=48, kl=kl, vl=vl, kg=kg, vg=vg, seed=vg)
        check_means(bt, 2, [1] * len(lens), offsets=False)


@pytest.mark.parametrize("B,heads,longest", [(1, 1, 20000), (3, 2, 9000), (70, 1, 700), (300, 2, 400), (700, 1, 90)])
def test_means_of_few_and_many_sequences(B, heads, longest):
    # from one sequence cut over the whole chip to more units than workgroups; more than 64
    # sequences are several of a lane's
    g = np.random.default_rng(B)
    lens = [int(x) for x in g.integers(0, longest, B)]
    lens[-1] = longest
    bt = Batch(lens, heads=heads, D=128, page=16, kg=64)
    check_means(bt, 1, [1] * B)


def test_means_of_even_lengths_past_one_share_each():
    # as many units as workgroups and more: the line is cut inside almost every unit
    bt = Batch([333] * 130, heads=4, D=64, page=32, kg=32)
    check_means(bt, 4, [1] * 130)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("share", [1, 5, 16, 20, 48, 50])
def test_means_of_chunks(D, share):
    counts, lens = [3, 70, 0, 1, 41], [1500, 70, 5, 900, 17]
    bt = Batch(lens, heads=1, D=D, page=16, vl=16, kg=64)
    check_means(bt, share, counts)


@pytest.mark.parametrize("D,share", [(64, 1), (128, 4), (256, 3)])
def test_means_of_a_long_chunk(D, share):
    bt = Batch([2500, 1024], heads=2, D=D, page=64, kg=64)
    check_means(bt, share, [1300, 1024], only=set(range(0, 2324, 7)) | {1299, 2323})


@pytest.mark.parametrize("D,share", [(64, 4), (128, 1), (128, 8), (256, 3)])
def test_means_of_trees(D, share):
    counts, lens = [7, 24, 0, 60, 33], [7, 600, 12, 61, 3000]
    bt = Batch(lens, heads=2, D=D, page=32, vl=16)
    check_means(bt, share, counts, tree_rows(counts, np.random.default_rng(D), 64))


def test_queries_that_precede_every_token():
    # more queries than tokens: the first ones stand before the cache's first token
    bt = Batch([5, 40, 0, 1], heads=2, D=64, page=16, kg=32)
    check_means(bt, 2, [9, 60, 3, 2])


def check_scores(bt, share, counts, tree=None, only=None, lowest=-8, highest=9):
    g = np.random.default_rng([len(counts), share])
    M, D = sum(counts), bt.D
    q = torch.from_numpy(g.integers(lowest, highest, (M, bt.heads * share, D)).astype(np.float32)).cuda().to(torch.bfloat16)
    scale = 6.0 / D ** 0.5 / (highest - lowest)
    out = as_f64(run(bt, q, counts, tree, out_dtype=torch.float16, scale=scale))
    k, v = decoded(bt)
    qr = ohd.rotate(as_f64(q).reshape(-1, D), 21).reshape(q.shape)
    scale = float(np.float32(scale))
    for m, b, mask in masks(bt, counts, tree):
        if (only is not None and m not in only) or not mask.any():
            continue
        for h in range(bt.heads * share):
            kk, vv = k[b][mask, h // share], v[b][mask, h // share]
            s = scale * (kk @ qr[m, h])
            p = np.exp(s - s.max())
            p /= p.sum()
            want = ohd.unrotate((p @ vv)[None], 22)[0]
            E = scale * (D + 16) * 2.0 ** -23 * (np.abs(kk) @ np.abs(qr[m, h])) + 2.0 ** -20 * np.abs(s).max()
            rel = np.expm1(2 * E.max()) + U + 64 * 2.0 ** -24 + len(s) * 2.0 ** -23
            room = (rel * np.linalg.norm(p @ np.abs(vv)) + 2.0 ** -32 * np.linalg.norm(np.abs(vv).sum(axis=0))
                    + U * 1.01 * np.linalg.norm(want) + 2.0 ** -25 * D ** 0.5)
            err = np.linalg.norm(out[m, h] - want)
            assert err <= room, (m, h, err / room)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kl,vl", [(256, 8), (16, 16), (4, 256), (8, 4)])
def test_scores_of_every_format(D, kl, vl):
    lens = [1, 2, 17, 100, 259, 1030]
    for kg in (32, 64, 128):
        bt = Batch(lens, heads=2, D=D, page=16, kl=kl, vl=vl, kg=kg, seed=kg)
        check_scores(bt, 3, [1] * len(lens))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("share", [1, 4])
def test_scores_of_chunks_and_trees(D, share):
    counts, lens = [3, 70, 41], [700, 70, 300]
    bt = Batch(lens, heads=2, D=D, page=16, kg=64)
    only = set(range(0, 114, 6)) | {2, 72, 113}
    check_scores(bt, share, counts, only=only)
    check_scores(bt, share, counts, tree_rows(counts, np.random.default_rng(3), 96), only=only)


def test_one_sided_queries_reach_large_scores():
    # integers of one sign: the rotated query's largest element is near the integers' limit
    bt = Batch([200, 31], heads=1, D=256, page=16, kg=64)
    check_scores(bt, 4, [1, 1], lowest=1, highest=9)


def test_no_table_at_all():
    bt = Batch([0, 0], heads=1, D=64, page=16, kg=32)
    q = torch.ones((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 3.0)
    tq.kv_attend(bt.cache, q, torch.tensor([5, 0], dtype=torch.int32, device="cuda"),
                 torch.empty((2, 0), dtype=torch.int32, device="cuda"), out=out)
    torch.cuda.synchronize()
    assert not out.any()


def test_empty_tensors_of_any_strides():
    bt = Batch([20], heads=1, D=64, page=16, kg=32)
    none = torch.empty(0, dtype=torch.bfloat16, device="cuda").as_strided((0, 1, 64), (1, 1, 2))
    slots = torch.empty(0, dtype=torch.int64, device="cuda")
    tq.kv_store(bt.cache, none, none, slots)
    lens, table = bt.dev()
    assert tq.kv_attend(bt.cache, none, lens, table, q_offsets=torch.zeros(2, dtype=torch.int32, device="cuda")).shape == none.shape
    assert tq.rope(none, slots, tq.rope_frequencies(64)).shape == none.shape
    k, v = tq.kv_load(bt.cache, slots)
    assert k.shape == v.shape == (0, 1, 64)
