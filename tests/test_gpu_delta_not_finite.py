"""What the gated delta rule does with values that are not finite."""
import math

import pytest
import torch

from test_gpu_delta import BF16, F32, call, inputs, on_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("H,T,at", [(2, 40, 0), (2, 300, 130), (90, 200, 199), (1, 1100, 777)])
def test_a_gate_that_is_not_a_number_shows(H, T, at, dt):
    # whole and in segments: NaN in its head from its token on and in the gradients before it, and nowhere else
    x = inputs(T, 2, H, H, T, 32, 24, dt)
    clean = call(on_gpu(x))
    x["g"][1, H - 1, at] = math.nan
    got = call(on_gpu(x))
    hit = torch.zeros(2, H, dtype=torch.bool)
    hit[1, H - 1] = True
    for n in clean:
        assert torch.equal(got[n][~hit], clean[n][~hit]), n
    for n in ("o", "dv", "dq", "dk", "dbeta", "dg"):
        assert torch.isnan(got[n][hit][:, at]).all(), n
    for n in ("h_final", "dh0"):
        assert torch.isnan(got[n][hit]).all(), n
    assert torch.isnan(got["o"][hit][:, at:]).all() and torch.isnan(got["dg"][hit][:, :at]).all()
    before = at // 64 * 64
    assert torch.equal(got["o"][hit][:, :before], clean["o"][hit][:, :before])
