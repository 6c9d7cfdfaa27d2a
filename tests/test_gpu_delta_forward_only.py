"""A forward-only call of the gated delta rule beside a training one: its o, too, is rounded to bf16 once (a half step of
2^-8, in the mean square 2^-8 / sqrt(3) of the value), by the bounds of test_gpu_delta.py for a training step's o."""
import pytest
import torch

from sequence_state_scan_amd import gla
from test_gpu_delta import BF16, inputs, near, on_gpu, reference, share

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,H,T,dk,dv,gates", [(2, 2, 300, 64, 64, "weak"), (1, 2, 700, 128, 128, "mid"), (1, 90, 70, 48, 72, "mid"),
                                               (1, 1, 2000, 32, 130, "zero")])
def test_forward_only_o_is_rounded_once(B, H, T, dk, dv, gates):
    x = inputs(T + 1, B, H, H, T, dk, dv, BF16, gates)
    r, c = reference(x), on_gpu(x)
    a = tuple(c[n] for n in ("q", "k", "v", "g", "beta"))
    o = gla.gla_delta_fwd(*a, h0=c["h0"], keep_saved=False)[0]
    near("o", o, r["o"], share("o", BF16, BF16))
    train = gla.gla_delta_fwd(*a, h0=c["h0"])[0]
    # before its rounding the two differ by the parts' own rounding alone: a step in one of 2^7 elements at most
    assert float((o != train).double().mean()) < 2.0 ** -7
