"""The gated delta rule in buffers that held something else, and in captured graphs whose inputs, lengths, slots and states
change between replays."""
import math

import pytest
import torch

from sequence_state_scan_amd import gla
from test_gpu_delta import BF16, F32, call, inputs, on_gpu

pytestmark = pytest.mark.gpu
NAMES = ("o", "h_final", "dq", "dk", "dv", "dg", "dbeta", "dh0")


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("H,Hk,T,dk,dv,lens", [(2, 1, 1500, 32, 40, (1500, 0, 1, 700)), (43, 43, 200, 60, 72, (200, 65, 64, 0)),
                                               (3, 3, 700, 100, 136, (1, 699, 128, 0)), (2, 2, 40, 24, 20, (0, 0, 0, 0))])
def test_buffers_full_of_nan_and_lengths(H, Hk, T, dk, dv, lens, dt):
    # whatever stands behind a sequence's end in the buffers between kernels is not read
    c = on_gpu(inputs(T, len(lens), H, Hk, T, dk, dv, dt, resets=2))
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    first = call(c, ln)
    a, dims = tuple(c[n] for n in ("q", "k", "v", "g", "beta")), (len(lens), H, Hk, T, dk, dv, dt)
    junk = lambda n: torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")  # noqa: E731  (NaN as floats)
    out = {n: torch.full_like(t, math.nan) for n, t in first.items()}
    o, h_final, saved = gla.gla_delta_fwd(*a, h0=c["h0"], lens=ln, o=out["o"], h_final=out["h_final"],
                                          saved=junk(gla.delta_saved_size(*dims)),
                                          workspace=junk(gla.delta_workspace_size(gla.GLA_FWD, *dims)))
    gla.gla_delta_bwd(*a, o, c["do"], saved, lens=ln, dhT=c["dhT"], workspace=junk(gla.delta_workspace_size(gla.GLA_BWD, *dims)),
                      **{n: out[n] for n in NAMES[2:]})
    for n in NAMES:
        assert torch.equal(first[n], out[n]), n
    only = gla.gla_delta_fwd(*a, h0=c["h0"], lens=ln, keep_saved=False,
                             workspace=junk(gla.delta_workspace_size(gla.GLA_FWD, *dims)))
    again = gla.gla_delta_fwd(*a, h0=c["h0"], lens=ln, keep_saved=False)
    assert torch.equal(only[0], again[0]) and torch.equal(only[1], again[1])


def captured(fn):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = fn()
    return graph, out


@pytest.mark.parametrize("T", [100, 1300])
def test_replays_with_other_lengths(T):
    x = [on_gpu(inputs(s, 3, 2, 1, T, 64, 48, BF16)) for s in range(3)]
    lens = [torch.tensor(n, dtype=torch.int32).cuda() for n in ((T, 1, 0), (0, T, 65), (64, T - 1, T + 5))]
    want = [call(c, n) for c, n in zip(x, lens)]
    held, ln = {n: t.clone() for n, t in x[0].items()}, lens[0].clone()
    graph, got = captured(lambda: call(held, ln))
    for turn in (2, 0, 1, 2, 0):
        for n in held:
            held[n].copy_(x[turn][n])
        ln.copy_(lens[turn])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n in got:
            assert torch.equal(got[n], want[turn][n]), (turn, n)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_replayed_tokens(dt):
    # a decoding loop: the graph of one token, with other slots and inputs every time
    B, H, Hk, dk, dv, steps = 5, 4, 2, 100, 72, 6
    c = on_gpu(inputs(9, B, H, Hk, steps, dk, dv, dt))
    names = ("q", "k", "v", "g", "beta")
    pool = torch.randn(9, H, dk, dv, generator=torch.Generator().manual_seed(3)).cuda()
    slots = [torch.randperm(9, generator=torch.Generator().manual_seed(s))[:B].to(torch.int32).cuda() for s in range(steps)]
    eager, want = pool.clone(), []
    for t in range(steps):
        want.append(gla.gla_delta_step(*(c[n][:, :, t:t + 1] for n in names), eager, slots=slots[t]))
    held, sl = [c[n][:, :, :1].contiguous() for n in names], slots[0].clone()
    scratch = pool.clone()
    graph, o = captured(lambda: gla.gla_delta_step(*held, scratch, slots=sl))
    scratch.copy_(pool)
    for t in range(steps):
        for h, n in zip(held, names):
            h.copy_(c[n][:, :, t:t + 1])
        sl.copy_(slots[t])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[t]), t
    assert torch.equal(scratch, eager)
