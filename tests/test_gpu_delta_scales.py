"""The gated delta rule with keys of any length.  With k and v times s_t, beta over s_t^2, the rule writes what it wrote: for
powers of two every product and sum is the same number, scaled, so that results are equal bit for bit."""
import pytest
import torch

from test_gpu_delta import BF16, F32, call, inputs, on_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("H,Hk,T,dk,dv", [(2, 1, 50, 32, 24), (2, 2, 700, 64, 80), (90, 90, 130, 100, 72)])
def test_keys_of_any_length(H, Hk, T, dk, dv, dt):
    x = inputs(T + 2, 1, H, Hk, T, dk, dv, dt, resets=2)
    want = call(on_gpu(x))
    s = torch.exp2(torch.randint(-9, 10, (T,), generator=torch.Generator().manual_seed(1)).double())
    y = dict(x, k=(x["k"] * s[:, None]).to(dt), v=(x["v"] * s[:, None]).to(dt), beta=(x["beta"] / s ** 2).float())
    got = call(on_gpu(y))
    s = s.cuda()
    for n, t in got.items():
        scale = {"dk": s[:, None], "dv": s[:, None], "dbeta": 1 / s ** 2}.get(n, 1)
        assert torch.equal((t.double() * scale).to(t.dtype), want[n]), n
