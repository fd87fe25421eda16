"""Calls of tq_verify and their answers in full, where a comparison by the oracle's clear decisions alone
would not see a wrong one."""

import numpy as np
import pytest
import torch

import rotation_lloyd_max_amd as tq
from test_gpu_verify import DTS, case, on_gpu, reference

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
