"""The gated delta rule on sizes that take every one of its kernels (delta_shapes.py; test_delta_shapes.py holds the list to
that), against the float64 code and the bounds of test_gpu_delta.py."""
import pytest
import torch

import test_gpu_delta as rule
from delta_shapes import BF16, CASES, F32

pytestmark = pytest.mark.gpu
DT = {BF16: torch.bfloat16, F32: torch.float32}


@pytest.mark.parametrize("case", CASES, ids=str)
def test_delta_kernels(case):
    B, H, Hk, T, dk, dv, dt, lens = case
    x = rule.inputs(T + dk + dv, B, H, Hk, T, dk, dv, DT[dt], "weak" if T > 400 else "mid", resets=2 if lens else 0)
    rule.check(x, None if lens is None else torch.tensor(lens), str(case))
