"""The cut of the gated delta rule's calls, on the host: its buffers are what their regions add up to, and the cases of
test_gpu_delta_shapes.py take every kernel."""
import itertools

import pytest
import torch

from delta_shapes import BF16, CASES, F32, KINDS, forward_bytes, kind, saved_bytes
from sequence_state_scan_amd import gla

DT = {BF16: torch.bfloat16, F32: torch.float32}
SIZES = [(B, H, Hk, T, dk, dv) for (B, H, Hk), T, (dk, dv) in itertools.product(
    ((1, 1, 1), (1, 4, 4), (2, 6, 3), (1, 24, 8), (1, 86, 86), (3, 67, 1)), (1, 64, 65, 130, 700, 2048, 9999),
    ((1, 1), (32, 64), (33, 65), (64, 130), (100, 200), (128, 128), (128, 1024)))]


@pytest.mark.parametrize("dt", [BF16, F32])
def test_buffers_hold_their_regions_and_no_more(dt):
    for s in SIZES + [c[:6] for c in CASES]:
        assert gla.delta_workspace_size(gla.GLA_FWD, *s, DT[dt]) == forward_bytes(*s, dt), s
        assert gla.delta_saved_size(*s, DT[dt]) == saved_bytes(*s, dt), s


def test_the_cases_take_every_kernel():
    assert {kind(B, H, T, dk, dv, dt) for B, H, Hk, T, dk, dv, dt, lens in CASES} == KINDS


def test_limits_as_documented():
    size = lambda B, H, T: gla.delta_saved_size(B, H, 1, T, 8, 8, torch.bfloat16)  # noqa: E731
    assert size(1, (1 << 18) - 1, 16 * 64) > 0 and size(2, 1, 64 * ((1 << 21) - 1)) > 0
    for B, H, T in ((1, 1 << 18, 1), (1 << 10, 1 << 8, 64), (2, 1, 64 * ((1 << 21) - 1) + 1), (1, 1 << 17, 64 * 32)):
        with pytest.raises(gla.GLAError):
            size(B, H, T)
