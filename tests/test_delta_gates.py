"""The bound on the gated delta rule's dg, on the host: it lets the sums in 64 bits pass, and refuses an o or a dv that is
only good to 12 bits, beside bf16 inputs to 10."""
import pytest
import torch

from delta_gates import gate_terms, gates_from
from test_gpu_delta import BF16, F32, inputs, near, reference, share

SIZES = [(2, 2, 1, 300, 16, 16), (1, 2, 2, 330, 48, 40)]


def rounded(t, bits):
    m, e = torch.frexp(t)
    return torch.ldexp((m * 2.0 ** bits).round() / 2.0 ** bits, e)


@pytest.mark.parametrize("gates", ["mid", "weak"])
@pytest.mark.parametrize("B,H,Hk,T,dk,dv", SIZES)
def test_bound_of_dg(B, H, Hk, T, dk, dv, gates):
    x = inputs(T + 1, B, H, Hk, T, dk, dv, F32, gates)
    r = reference(x)
    terms = gate_terms(x, r)
    near("dg", gates_from(x, r["o"], r["dv"]), r["dg"], 1e-12, terms)
    for dt, bits in ((F32, 12), (BF16, 10)):
        for o, dval in ((rounded(r["o"], bits), r["dv"]), (r["o"], rounded(r["dv"], bits))):
            with pytest.raises(AssertionError, match="dg"):
                near("dg", gates_from(x, o, dval), r["dg"], share("dg", dt, F32), terms)
