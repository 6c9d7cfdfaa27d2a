"""The gated delta rule's dg against the size of what it is summed from (delta_gates.py), several times closer than the
products of norms that test_gpu_delta.py takes for it."""
import pytest

from delta_gates import gate_terms
from test_gpu_delta import BF16, F32, call, inputs, near, on_gpu, reference, share

pytestmark = pytest.mark.gpu
SIZES = [(2, 2, 1, 512, 16, 16), (1, 2, 2, 600, 64, 48), (1, 2, 1, 512, 128, 128), (1, 17, 17, 300, 100, 72), (2, 1, 1, 40, 8, 200)]


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("gates", ["mid", "weak", "strong", "mixed"])
@pytest.mark.parametrize("B,H,Hk,T,dk,dv", SIZES)
def test_dg_by_its_own_terms(B, H, Hk, T, dk, dv, gates, dt):
    x = inputs(T + dk, B, H, Hk, T, dk, dv, dt, gates)
    r = reference(x)
    near("dg", call(on_gpu(x))["dg"], r["dg"], share("dg", dt, F32), gate_terms(x, r))
