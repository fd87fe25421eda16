"""Calls of tq_verify and their answers in full, where a comparison by the oracle's clear decisions alone
would not see a wrong one."""

import numpy as np
import pytest
import torch

import rotation_lloyd_max_amd as tq
from test_gpu_verify import CLEAR, DTS, case, on_gpu, reference

pytestmark = pytest.mark.gpu
CODES = {"fp32": tq.F32, "bf16": tq.BF16, "fp16": tq.F16}


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("tdt,ddt", [("bf16", "fp32"), ("fp32", "fp16"), ("bf16", "bf16"), ("fp16", None)])
def test_a_step_of_no_rows_keeps_nothing(tdt, ddt, tree):
    # through the C interface, whose arrays may be longer than the step: 0 rows of 3 sequences
    x, y = (torch.zeros((2, 100), dtype=DTS[n or "fp32"], device="cuda") for n in (tdt, ddt))
    i32 = lambda n, v: torch.full((n,), v, dtype=torch.int32, device="cuda")  # noqa: E731
    kept, out, path, words = i32(3, 1234), i32(2, 1234), i32(2, 1234), i32(4, 0)
    rc = tq.lib().tq_verify(x.data_ptr(), CODES[tdt], 100, y.data_ptr() if ddt else None, CODES[ddt or "fp32"], 100, 0, 100, 3,
                            words.data_ptr(), 0, words.data_ptr(), words.data_ptr() if tree else None, x.data_ptr(), None,
                            kept.data_ptr(), out.data_ptr(), path.data_ptr(), None, 0, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0 and kept.tolist() == [0, 0, 0]
    assert out.tolist() == path.tolist() == [1234, 1234]


def steady(n, drafted, tree):
    """A sequence of n rows of even probabilities over 50 tokens, row i drafting token i % 50; 0.01 as its number
    lets a row stay, 1.0 turns it away (and a draft's too, whose probabilities are the same)."""
    even = torch.full((n, 50), 0.02)
    return dict(target=even, tokens=np.arange(n) % 50, uniforms=np.full(n, 0.01, np.float32), offsets=np.array([0, n]),
                draft=even.clone() if drafted else None, parents=np.maximum(np.arange(n) - 1, 0) if tree else None, temperature=None,
                target_kind="probabilities", draft_kind="probabilities")


def answers(c):
    got = tq.verify(**on_gpu(c))
    kept, tokens, path, _ = reference(c)
    torch.cuda.synchronize()
    assert got.kept.tolist() == kept.tolist() and got.path.tolist() == path.tolist()
    assert got.tokens.tolist() == tokens.tolist()
    k = got.kept.item()
    return k, got.tokens[k - 1].item()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("drafted", [False, True])
@pytest.mark.parametrize("tree", [False, True])
def test_a_drafted_tokens_probability_is_none(bad, drafted, tree):
    # the row makes no distribution: its child does not stay, whatever its number, and the new token is -1
    for n, row in ((2, 0), (6, 3), (70, 64), (300, 254), (300, 255), (300, 256), (300, 280)):
        for name in ("target", "draft") if drafted else ("target",):
            for u in (0.01, 0.0, 1.0):
                c = steady(n, drafted, tree)
                c[name][row, (row + 1) % 50] = bad
                c["uniforms"][row + 1] = u
                assert answers(c) == (row + 1, -1)
    # at a token that nobody looks at
    c = steady(6, drafted, tree)
    c["target"][2, 9] = bad
    k, new = answers(c)
    assert k == 6 and new >= 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("drafted", [False, True])
def test_one_of_several_siblings_probability_is_none(bad, drafted):
    for place in range(4):
        c = steady(5, drafted, True)
        c["parents"] = np.zeros(5, np.int64)
        c["target"][0, 1 + place] = bad
        c["uniforms"][1:] = 1.0
        assert answers(c) == (1, -1)       # all are turned away, the bad one among them
        if place:
            c["uniforms"][1] = 0.01
            assert answers(c)[0] == 2      # the first stays: the others are not looked at
        c["uniforms"][1:] = 1.0
        c["uniforms"][4] = 0.0             # the last would stay
        assert answers(c) == (1, -1)


@pytest.mark.parametrize("V", [8191, 8192, 16385, 50257])
@pytest.mark.parametrize("tree,ddt", [(False, "bf16"), (True, "fp16"), (True, None), (False, None)])
@pytest.mark.parametrize("kind", ["logits", "probabilities"])
def test_rows_around_the_ends_of_pieces(V, tree, ddt, kind):
    # every sequence has rows and clear decisions, and all are compared
    for seed, B, most in ((60, 1, 2), (61, 2, 5), (62, 3, 3)):
        c = case(seed, B, most, V, "fp32", ddt, kind, tree, ragged=False)
        assert len(c["tokens"]) == B * most
        want = reference(c)
        assert (want[3] > CLEAR).all()
        got = tq.verify(**on_gpu(c))
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert x.tolist() == y.tolist()
