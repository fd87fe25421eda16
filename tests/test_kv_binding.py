"""Calls of the serving binding that must be refused, or must not be: gradients, overlapping outputs, index
values beyond 32 bits. CPU tensors, so that every check is shown to come before the library."""

import os

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
