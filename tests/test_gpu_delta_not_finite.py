"""What the gated delta rule does with values that are not finite."""
import math

import pytest
import torch

from sequence_state_scan_amd import gla
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


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("held", [math.nan, math.inf])
@pytest.mark.parametrize("H,T", [(2, 50), (2, 300), (90, 70), (1, 1100)])
def test_a_first_tokens_reset_drops_what_h0_holds(H, T, held, dt):
    # a state of a pool that is used again; the empty sequence's state is h0 all the same
    x = inputs(T, 3, H, H, T, 32, 24, dt)
    x["g"][:, :, 0] = -math.inf
    lens = torch.tensor([T, 0, max(1, T // 2)], dtype=torch.int32).cuda()
    x["h0"] = None
    want = call(on_gpu(x), lens)
    a = [x[n].cuda() for n in ("q", "k", "v", "g", "beta")]
    only = gla.gla_delta_fwd(*a, lens=lens, keep_saved=False)
    x["h0"] = torch.full((3, H, 32, 24), held)
    got = call(on_gpu(x), lens)
    again = gla.gla_delta_fwd(*a, h0=x["h0"].cuda(), lens=lens, keep_saved=False)
    for n in want:
        if n == "h_final":
            assert torch.equal(got[n][[0, 2]], want[n][[0, 2]]) and not torch.isfinite(got[n][1]).any()
        else:
            assert torch.equal(got[n], want[n]), n
    assert torch.equal(again[0], only[0]) and torch.equal(again[1][[0, 2]], only[1][[0, 2]])
    # the calls for single tokens and for chunks agree
    pool = x["h0"].cuda()
    o = gla.gla_delta_step(*(t[:, :, :1] for t in a), pool)
    one, state, _ = gla.gla_delta_fwd(*(t[:, :, :1] for t in a), h0=x["h0"].cuda(), keep_saved=False)
    assert torch.isfinite(o).all() and torch.isfinite(pool).all() and torch.isfinite(one).all() and torch.isfinite(state).all()
