"""Layer norm where a workgroup has several rows one after the other: the row loaded ahead, the reload of wide rows, the step
from one batch element to the next and the halves of LDS used in turn, against float64 by the bounds of test_gpu_delta.py."""
import pytest
import torch

from sequence_state_scan_amd import gla
from test_gpu_delta import BF16, F32, norm_check, norm_reference

pytestmark = pytest.mark.gpu

# rows for at least two passes of every workgroup, forward (1024 of 256 lanes) and backward (half as many), none a multiple
# of the step: 16 rows a workgroup, 2, 1, and rows of 512 lanes with 1, 2 and 4 slots a lane, whole slots and not
SIZES = [(2, 17001, 96), (2, 9000, 95), (3, 1401, 1000), (2, 1300, 2048), (3, 701, 2051), (3, 400, 5000), (3, 400, 8191),
         (3, 403, 12345), (2, 600, 16384)]


def wide_view(t, off):
    """The same values as a slice of wider rows, off 16 bytes."""
    B, T, D = t.shape
    pool = torch.full((B, T + 2, D + off + 3), float("nan"), dtype=t.dtype, device="cuda")
    v = pool[:, 1:T + 1, off:off + D]
    v.copy_(t)
    return v


@pytest.mark.parametrize("dt,st", [(F32, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("B,T,D", SIZES)
def test_many_rows_a_workgroup(B, T, D, dt, st):
    gen = torch.Generator().manual_seed(D)
    rnd = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    x, dn, residual, d_out = (rnd(B, T, D) + 1).to(dt), rnd(B, T, D).to(dt), (2 * rnd(B, T, D)).to(st), rnd(B, T, D).to(st)
    w, b = 1 + 0.1 * rnd(D), 0.1 * rnd(D)
    ref = norm_reference(x, w, b, residual, 1e-5, dn, d_out)
    xg, wg, bg = wide_view(x, 1), w.cuda(), b.cuda()
    rg = residual.cuda().transpose(0, 1).contiguous().transpose(0, 1)  # rows of the batch side by side
    f = gla.gla_layernorm_fwd(xg, wg, bg, residual=rg)
    g = gla.gla_layernorm_bwd(xg, f, wide_view(dn, 2), wg, d_out=wide_view(d_out, 5), residual=rg)
    norm_check("%d x %d" % (B * T, D), {"out": f["out"], "normed": f["normed"], **g}, ref, B * T, D)
    # the same in the residual's place, and of contiguous tensors
    stream = residual.cuda()
    c = gla.gla_layernorm_fwd(x.cuda(), wg, bg, residual=stream, out=stream, keep_stats=False)
    assert c["out"] is stream and torch.equal(stream, f["out"]) and torch.equal(c["normed"], f["normed"])
    # the norm alone
    ref = norm_reference(x, w, None, None, 1e-5, dn)
    f = gla.gla_layernorm_fwd(x.cuda(), wg)
    g = gla.gla_layernorm_bwd(x.cuda(), f, dn.cuda(), wg, bias=False)
    norm_check("alone", {"normed": f["normed"], "dx": g["dx"], "dw": g["dw"]}, ref, B * T, D)
