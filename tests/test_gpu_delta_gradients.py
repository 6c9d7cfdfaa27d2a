"""dq and dk of the gated delta rule where no state enters or leaves a chunk (documents of a chunk each, no h0, no dhT): of
what they are computed from nothing is rounded to one bf16 then, and they themselves once, by the bounds of test_gpu_delta.py
for dv."""
import math

import pytest
import torch

from test_gpu_delta import BF16, call, inputs, near, on_gpu, reference, share

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gates", ["mid", "weak", "zero"])
@pytest.mark.parametrize("B,H,Hk,T,dk,dv", [(2, 4, 2, 256, 64, 64), (1, 3, 3, 300, 128, 128), (1, 40, 40, 64, 32, 100),
                                            (3, 2, 1, 200, 100, 200)])
def test_gradients_inside_a_chunk_are_rounded_once(B, H, Hk, T, dk, dv, gates):
    x = inputs(T + 3, B, H, Hk, T, dk, dv, BF16, gates)
    x["g"][:, :, ::64] = -math.inf
    x["h0"] = x["dhT"] = None
    r, got = reference(x), call(on_gpu(x))
    for n in ("dq", "dk"):
        near(n, got[n], r[n], share("dv", BF16, BF16))
