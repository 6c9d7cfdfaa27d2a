"""The recurrent-block operators (gla_recur_*, gla_join_*, gla_step) against plain float64 code
written from their formulas.

Tolerances are error bounds, element by element, with u = 2^-24 (half a float32 step) and
eps(dtype)/2 for the rounding of the output:
  - a = exp(g) through the base-2 exponential is off by at most (3 + 2|g|) u relative (the product
    with log2 e, its constant, one step of the instruction), and every multiply-add or product of
    decays adds u, so a term that crosses a token gains at most (5 + 2|g|) u: the bound on the
    state is u times  W_t = a_t (W_{t-1} + (5 + 2|g_t|) H_{t-1}),  H the recurrence over |terms|,
    plus 8 u H for the terms themselves (input factor and product);
  - a norm's mean of squares sums positive terms, off by the number of additions in a chain times
    u; the chains here (a lane's few, the lanes' six, the waves' sixteen) are below 48; each
    gradient is bounded by the same formula over absolute values times 64 u (+ 4 max|z| u for
    the gate's exponential), and a sum over N rows by its longest chain more.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from sequence_state_scan_amd import gla, inputs

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


def half_step(dt):
    return torch.finfo(dt).eps / 2 if dt != F32 else U


def rnd(gen, *shape):
    return torch.randn(shape, generator=gen, dtype=torch.float64)


def inside(name, got, ref, tol):
    """|got - ref| <= tol everywhere, on the CPU in float64."""
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert torch.isfinite(got).all(), "%s: not finite" % name
    over = (got - ref).abs() - tol
    i = int(over.argmax()) if over.numel() else 0
    assert over.numel() == 0 or float(over.max()) <= 0, "%s: off by %.3e at %d where %.3e is allowed (value %.3e)" % (
        name, float((got - ref).abs().flatten()[i]), i, float(torch.as_tensor(tol).expand_as(ref).flatten()[i]),
        float(ref.flatten()[i]))


# ---------------------------------------------------------------------------------- recurrence

def factor(g, mode):
    if mode == "plain":
        return torch.ones_like(g), torch.zeros_like(g)
    if mode == "lerp":
        return -torch.expm1(g), -torch.exp(g)
    b = torch.sqrt(-torch.expm1(2 * g))
    return b, torch.where(b > 0, -torch.exp(2 * g) / b, torch.zeros_like(b))


def recur_reference(x, g, h0, lens, mode, dh=None, dhT=None):
    """Token by token in float64: values and error bounds (before the outputs' rounding)."""
    B, T, D = x.shape
    a = torch.exp(g)
    beta, slope = factor(g, mode)
    hop = torch.where(a > 0, 5 + 2 * g.abs(), torch.zeros_like(a))
    h, H, W = h0.clone(), h0.abs(), torch.zeros_like(h0)
    hs, tols, before, tol_before = (torch.zeros_like(x) for _ in range(4))
    for t in range(T):
        live = (t < lens)[:, None]
        before[:, t], tol_before[:, t] = h, U * (8 * H + W)
        at = a[:, t]
        nh = at * h + beta[:, t] * x[:, t]
        nW = at * (W + torch.where(at > 0, hop[:, t] * H, 0.0))
        nH = at * H + (beta[:, t] * x[:, t]).abs()
        h, H, W = torch.where(live, nh, h), torch.where(live, nH, H), torch.where(live, nW, W)
        hs[:, t] = torch.where(live, h, 0.0)
        tols[:, t] = torch.where(live, U * (8 * H + W), 0.0)
    r = {"h": (hs, tols), "h_final": (h, U * (8 * H + W))}
    if dh is None:
        return r
    G, GH, GW = dhT.clone(), dhT.abs(), torch.zeros_like(dhT)
    z = {n: torch.zeros_like(x) for n in ("dx", "dx_tol", "dg", "dg_tol")}
    for t in range(T - 1, -1, -1):
        live = (t < lens)[:, None]
        D_, DH = G + dh[:, t], GH + dh[:, t].abs()
        tolD = U * (8 * DH + GW)
        z["dx"][:, t] = torch.where(live, beta[:, t] * D_, 0.0)
        z["dx_tol"][:, t] = torch.where(live, beta[:, t] * (tolD + 8 * U * DH), 0.0)
        at, hb, th, sx = a[:, t], before[:, t].abs(), tol_before[:, t], (slope[:, t] * x[:, t]).abs()
        z["dg"][:, t] = torch.where(live, at * before[:, t] * D_ + slope[:, t] * x[:, t] * D_, 0.0)
        z["dg_tol"][:, t] = torch.where(live, at * (hb * tolD + th * DH + hop[:, t] * U * hb * DH) +
                                        sx * (tolD + (16 + 4 * g[:, t].abs().nan_to_num(posinf=0)) * U * DH), 0.0)
        nW = at * (GW + torch.where(at > 0, hop[:, t] * DH, 0.0))
        G, GH, GW = torch.where(live, at * D_, G), torch.where(live, at * DH, GH), torch.where(live, nW, GW)
    r.update(dx=(z["dx"], z["dx_tol"]), dg=(z["dg"], z["dg_tol"]), dh0=(G, U * (8 * GH + GW)))
    return r


def recur_inputs(seed, B, T, D, dt, gates="mid", resets=0):
    gen = torch.Generator().manual_seed(seed)
    x, dh = rnd(gen, B, T, D).to(dt), rnd(gen, B, T, D).to(dt)
    pre = rnd(gen, B, T, D)
    g = {"mid": lambda: torch.nn.functional.logsigmoid(pre) / 4, "weak": lambda: -pre.abs() / 512,
         "strong": lambda: -8 * pre.abs(), "zero": lambda: 0 * pre}[gates]().float()
    if resets:
        g[:, torch.randint(0, T, (resets,), generator=gen)] = -math.inf
    h0, dhT = rnd(gen, B, D).float(), rnd(gen, B, D).float()
    return x, g, dh, h0, dhT


def check_recur(x, g, dh, h0, dhT, lens, mode, label, wrap=lambda t: t.cuda()):
    B, T, D = x.shape
    gpu = lambda t: None if t is None else t.cuda()  # noqa: E731
    full = torch.full((B,), T) if lens is None else lens.clamp(0, T)
    zero = torch.zeros(B, D, dtype=torch.float64)
    r = recur_reference(x.double(), g.double(), zero if h0 is None else h0.double(), full, mode, dh.double(),
                        zero if dhT is None else dhT.double())
    ln = None if lens is None else lens.to(torch.int32).cuda()
    xc, gc, dc = wrap(x), wrap(g), wrap(dh)
    h, chunk_in, h_final = gla.gla_recur_fwd(xc, gc, h0=gpu(h0), lens=ln, mode=mode)
    dx, dg, dh0 = gla.gla_recur_bwd(xc, gc, dc, chunk_in, lens=ln, dhT=gpu(dhT), mode=mode)
    torch.cuda.synchronize()
    for n, t in (("h", h), ("h_final", h_final), ("dx", dx), ("dg", dg), ("dh0", dh0)):
        ref, tol = r[n]
        inside(label + " " + n, t, ref, tol + half_step(t.dtype) * ref.abs() + half_step(t.dtype) * tol)
    return h, chunk_in, h_final, dx, dg, dh0


SIZES = [(1, 1, 1), (3, 1, 64), (2, 2, 7), (1, 16, 130), (2, 127, 64), (1, 128, 256), (2, 129, 65), (5, 300, 24),
         (1, 777, 100), (2, 1025, 33), (1, 2048, 8)]


@pytest.mark.parametrize("mode", ["plain", "lerp", "norm"])
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("B,T,D", SIZES)
def test_recur_against_the_formulas(B, T, D, dt, mode):
    x, g, dh, h0, dhT = recur_inputs(B * 1000 + T, B, T, D, dt)
    check_recur(x, g, dh, h0, dhT, None, mode, "B%d T%d D%d" % (B, T, D))


@pytest.mark.parametrize("gates", ["weak", "strong", "zero"])
@pytest.mark.parametrize("mode", ["plain", "lerp", "norm"])
def test_recur_gates(gates, mode):
    x, g, dh, h0, dhT = recur_inputs(7, 2, 400, 96, F32, gates)
    check_recur(x, g, dh, h0, dhT, None, mode, gates)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("D", [64, 41])
def test_recur_lengths_and_what_stands_behind_them(dt, D):
    # lengths of zero and one, a full one, and values outside 0..T; NaN and infinities behind the ends
    T = 333
    lens = torch.tensor([0, 1, T, 128, 129, 200, -3, T + 9])
    x, g, dh, h0, dhT = recur_inputs(3, len(lens), T, D, dt)
    clean = check_recur(x, g, dh, h0, dhT, lens, "norm", "lens")
    for b, n in enumerate(lens.clamp(0, T).tolist()):
        x[b, n:], g[b, n:], dh[b, n:] = math.nan, math.inf, math.nan
    ln = lens.to(torch.int32).cuda()
    h, chunk_in, h_final = gla.gla_recur_fwd(x.cuda(), g.cuda(), h0=h0.cuda(), lens=ln, mode="norm")
    dirty = (h, chunk_in, h_final) + gla.gla_recur_bwd(x.cuda(), g.cuda(), dh.cuda(), chunk_in, lens=ln, dhT=dhT.cuda(),
                                                       mode="norm")
    for a, b in zip(clean, dirty):
        assert torch.equal(a, b)


def test_recur_resets_cut_documents_apart():
    B, T, D = 2, 700, 96
    x, g, dh, h0, dhT = recur_inputs(11, B, T, D, F32, resets=6)
    for mode in ("plain", "lerp", "norm"):
        check_recur(x, g, dh, h0, dhT, None, mode, "resets " + mode)
    # a document's results do not depend on what stands before its reset, not even NaN
    cut = 300
    g[:, cut] = -math.inf
    ref = gla.gla_recur_fwd(x.cuda(), g.cuda(), mode="plain")[0]
    x[:, cut - 1] = math.nan
    got = gla.gla_recur_fwd(x.cuda(), g.cuda(), mode="plain")[0]
    assert torch.equal(got[:, cut:], ref[:, cut:]) and torch.isnan(got[:, cut - 1]).all()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("off,pad", [(0, 64), (3, 5), (8, 8), (1, 0)])
def test_recur_views(dt, off, pad):
    # x, g and dh as slices of wider rows, at every alignment; a batch that is expanded
    B, T, D = 3, 260, 64
    x, g, dh, h0, dhT = recur_inputs(5, B, T, D, dt)

    def wrap(t):
        wide = torch.full((B, T + 2, off + D + pad), math.nan, dtype=t.dtype, device="cuda")
        wide[:, 1:T + 1, off:off + D] = t.cuda()
        return wide[:, 1:T + 1, off:off + D]

    a = check_recur(x, g, dh, h0, dhT, None, "lerp", "views", wrap)
    b = check_recur(x, g, dh, h0, dhT, None, "lerp", "contiguous")
    for s, t in zip(a, b):
        assert torch.equal(s, t)
    one = x[:1].cuda().expand(B, T, D)
    assert torch.equal(gla.gla_recur_fwd(one, g.cuda())[0], gla.gla_recur_fwd(one.contiguous(), g.cuda())[0])


def test_recur_gradients_against_differences():
    # float64 differences of the float64 recurrence, so that the formulas themselves are tested
    B, T, D = 1, 9, 5
    for mode in ("plain", "lerp", "norm"):
        x, g, dh, h0, dhT = (t.double() for t in recur_inputs(2, B, T, D, F32))
        lens = torch.full((B,), T)

        def loss(x, g, h0):
            r = recur_reference(x, g, h0, lens, mode)
            return float((r["h"][0] * dh).sum() + (r["h_final"][0] * dhT).sum())

        r = recur_reference(x, g, h0, lens, mode, dh, dhT)
        for n, at in (("dx", 0), ("dg", 1), ("dh0", 2)):
            args = [x, g, h0]
            for i in range(0, args[at].numel(), 7):
                step = torch.zeros_like(args[at])
                step.view(-1)[i] = 1e-6
                hi, lo = (loss(*(a + s * step if k == at else a for k, a in enumerate(args))) for s in (1, -1))
                want = float(r[n][0].reshape(-1)[i])
                assert abs((hi - lo) / 2e-6 - want) <= 1e-6 * (1 + abs(want)), (mode, n, i)


def test_recur_forward_only_and_given_buffers():
    x, g, _, h0, _ = recur_inputs(1, 2, 300, 72, BF16)
    a = gla.gla_recur_fwd(x.cuda(), g.cuda(), h0=h0.cuda())
    b = gla.gla_recur_fwd(x.cuda(), g.cuda(), h0=h0.cuda(), keep_chunk_states=False)
    assert b[1] is None and torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])
    out = [torch.full_like(t, math.nan) for t in a]
    c = gla.gla_recur_fwd(x.cuda(), g.cuda(), h0=h0.cuda(), h=out[0], chunk_in=out[1], h_final=out[2])
    assert all(s is t and torch.equal(s, u) for s, t, u in zip(c, out, a))


def test_recur_is_the_same_every_time():
    x, g, dh, h0, dhT = (t.cuda() for t in recur_inputs(8, 1, 20000, 256, BF16))
    first = None
    for _ in range(5):
        h, chunk_in, h_final = gla.gla_recur_fwd(x, g, h0=h0, mode="norm")
        res = (h, chunk_in, h_final) + gla.gla_recur_bwd(x, g, dh, chunk_in, dhT=dhT, mode="norm")
        first = first or res
        for s, t in zip(first, res):
            assert torch.equal(s, t)


@pytest.mark.parametrize("T,D", [(40000, 72), (9000, 1024)])
def test_recur_long(T, D):
    x, g, dh, h0, dhT = recur_inputs(4, 1, T, D, BF16, "weak")
    check_recur(x, g, dh, h0, dhT, None, "norm", "T%d" % T)


@pytest.mark.parametrize("mode", ["plain", "lerp", "norm"])
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("B,D", [(1, 1), (1, 2048), (5, 100), (70, 264), (300, 24)])
def test_recur_step(B, D, dt, mode):
    x, g, _, _, _ = recur_inputs(B + D, B, 1, D, dt)
    gen = torch.Generator().manual_seed(B)
    pool = rnd(gen, B + 3, D).float()
    slots = torch.randperm(B + 3, generator=gen)[:B].to(torch.int32)
    if B > 2:
        slots[1] = -1
    state = pool.cuda()
    h = gla.gla_recur_step(x[:, 0].cuda(), g[:, 0].cuda(), state, slots=slots.cuda(), mode=mode)
    want = pool.double()
    for b in range(B):
        s = int(slots[b])
        if s < 0:
            assert not h[b].any()
            continue
        r = recur_reference(x[b:b + 1].double(), g[b:b + 1].double(), pool[s:s + 1].double(), torch.ones(1), mode)
        ref, tol = r["h_final"]
        inside("state", state[s:s + 1], ref, tol + U * ref.abs())
        inside("h", h[b:b + 1], ref, (tol + half_step(dt) * ref.abs()) * (1 + half_step(dt)))
        want[s] = state[s].cpu().double()
    assert torch.equal(state.cpu().double(), want)  # the other states stand as they were


def test_recur_step_continues_a_prompt():
    x, g, _, h0, _ = recur_inputs(12, 3, 131, 80, F32)
    x, g, h0 = x.cuda(), g.cuda(), h0.cuda()
    h, _, state = gla.gla_recur_fwd(x[:, :129], g[:, :129], h0=h0, mode="lerp")
    whole, _, last = gla.gla_recur_fwd(x, g, h0=h0, mode="lerp")
    for t in (129, 130):
        s = gla.gla_recur_step(x[:, t], g[:, t], state, mode="lerp")
        assert torch.allclose(s, whole[:, t], rtol=1e-5, atol=1e-6)
    assert torch.allclose(state, last, rtol=1e-5, atol=1e-6)


def test_bad_slots_give_nan_and_touch_nothing():
    x, g, _, _, _ = recur_inputs(1, 6, 1, 48, F32)
    pool = torch.randn(4, 48, device="cuda")
    slots = torch.tensor([2, 4, 2, 0, -7, 1 << 30], dtype=torch.int32, device="cuda")
    state = pool.clone()
    h = gla.gla_recur_step(x[:, 0].cuda(), g[:, 0].cuda(), state, slots=slots)
    assert torch.isnan(h[[1, 2, 5]]).all() and torch.isfinite(h[[0, 3, 4]]).all() and not h[4].any()
    assert torch.equal(state[[1, 3]], pool[[1, 3]]) and torch.equal(state[2], h[0]) and torch.equal(state[0], h[3])
    q = torch.randn(6, 2, 3, 16, device="cuda")
    v = torch.randn(6, 2, 3, 24, device="cuda")
    pool = torch.randn(4, 2, 16, 24, device="cuda")
    state = pool.clone()
    o = gla.gla_step(q, q, v, -q.abs(), state, slots=slots)
    assert torch.isnan(o[[1, 2, 5]]).all() and torch.isfinite(o[[0, 3, 4]]).all() and not o[4].any()
    assert torch.equal(state[[1, 3]], pool[[1, 3]]) and not torch.equal(state[[0, 2]], pool[[0, 2]])


def test_a_slot_named_twice_far_apart():
    B, D = 300, 40
    x, g, _, _, _ = recur_inputs(2, B, 1, D, F32)
    x, g = x[:, 0].cuda(), g[:, 0].cuda()
    slots = torch.randperm(400, generator=torch.Generator().manual_seed(3))[:B].to(torch.int32)
    bad = {70: 3, 199: 64, 299: 0, 200: 199}  # 200 repeats 199's, which is 64's: both later ones are refused
    for i, j in bad.items():
        slots[i] = slots[j]
    pool = torch.randn(400, D, device="cuda")
    state = pool.clone()
    h = gla.gla_recur_step(x, g, state, slots=slots.cuda())
    good = [i for i in range(B) if i not in bad]
    assert torch.isnan(h[list(bad)]).all() and torch.isfinite(h[good]).all()
    want = pool.clone()
    rows = slots[good].long().cuda()
    sub = pool[rows].clone()
    assert torch.equal(gla.gla_recur_step(x[good], g[good], sub), h[good])
    want[rows] = sub
    assert torch.equal(state, want)


# ---------------------------------------------------------------------------------------- step

def step_reference(q, k, v, g, S):
    """Token by token in float64; error bounds of o and S as for the recurrence, o's sum of dk terms
    of either sign adding its longest chain (dk / 16 in a lane, then 4 exchanges and sums)."""
    B, H, n, dk = q.shape
    M, W = S.abs(), torch.zeros_like(S)
    os, tols = [], []
    for t in range(n):
        a = torch.exp(g[:, :, t])[..., None]
        kv = k[:, :, t, :, None] * v[:, :, t, None, :]
        W = a * (W + torch.where(a > 0, (5 + 2 * g[:, :, t, :, None].abs()) * M, torch.zeros_like(M)))
        S, M = a * S + kv, a * M + kv.abs()
        qt = q[:, :, t, :, None]
        os.append((qt * S).sum(2))
        tols.append((qt.abs() * U * (8 * M + W + (24 + dk / 16) * M)).sum(2))
    return torch.stack(os, 2), torch.stack(tols, 2), S, U * (8 * M + W)


def step_inputs(seed, B, H, n, dk, dv, dt):
    gen = torch.Generator().manual_seed(seed)
    q, k, v = rnd(gen, B, H, n, dk).to(dt), rnd(gen, B, H, n, dk).to(dt), rnd(gen, B, H, n, dv).to(dt)
    g = (torch.nn.functional.logsigmoid(rnd(gen, B, H, n, dk)) / 4).float()
    return q, k, v, g, rnd(gen, B + 2, H, dk, dv).float()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("B,H,n,dk,dv", [(1, 1, 1, 1, 1), (1, 4, 1, 128, 256), (3, 2, 1, 64, 64), (2, 3, 5, 100, 96),
                                         (2, 1, 2, 33, 17), (1, 2, 9, 16, 66), (2, 2, 1, 256, 40), (40, 2, 1, 32, 32),
                                         (1, 1, 3, 129, 260)])
def test_step(B, H, n, dk, dv, dt):
    q, k, v, g, pool = step_inputs(dk + dv, B, H, n, dk, dv, dt)
    g[0, 0, n - 1, 0] = -math.inf
    slots = torch.randperm(B + 2, generator=torch.Generator().manual_seed(1))[:B]
    state = pool.cuda()
    o = gla.gla_step(q.cuda(), k.cuda(), v.cuda(), g.cuda(), state, slots=slots.to(torch.int32).cuda())
    ref, tol, S, tolS = step_reference(q.double(), k.double(), v.double(), g.double(), pool[slots].double())
    inside("o", o, ref, (tol + half_step(dt) * ref.abs()) * (1 + half_step(dt)))
    inside("state", state[slots.cuda()], S, tolS + U * S.abs())
    rest = [i for i in range(B + 2) if i not in slots.tolist()]
    assert torch.equal(state[rest].cpu(), pool[rest])


def test_step_views_and_unaligned_rows():
    # q, k, v, g cut out of one token-major projection, v starting off 8 bytes
    B, H, n, dk, dv = 2, 3, 4, 32, 64
    q, k, v, g, pool = step_inputs(3, B, H, n, dk, dv, BF16)
    a, s1, s2 = (pool.cuda() for _ in range(3))
    ref = gla.gla_step(q.cuda(), k.cuda(), v.cuda(), g.cuda(), s1)
    for off in (0, 1, 4):
        wide = torch.zeros(B, n, off + H * (2 * dk + dv), dtype=BF16, device="cuda")
        parts, at = [], off
        for t in (v, q, k):
            w = H * t.shape[-1]
            view = wide[:, :, at:at + w].unflatten(2, (H, t.shape[-1])).transpose(1, 2)
            view.copy_(t.cuda())
            parts.append(view)
            at += w
        s2 = a.clone()
        got = gla.gla_step(parts[1], parts[2], parts[0], g.transpose(1, 2).contiguous().transpose(1, 2).cuda(), s2)
        assert torch.equal(got, ref) and torch.equal(s2, s1)


def test_step_with_shared_heads():
    # one q, k and g for all heads, as expanded views
    B, H, n, dk, dv = 3, 4, 2, 48, 64
    q, k, v, g, pool = (t.cuda() for t in step_inputs(6, B, H, n, dk, dv, BF16))
    one = lambda t: t[:, :1].expand(B, H, n, dk)  # noqa: E731
    s1, s2 = pool.clone(), pool.clone()
    o = gla.gla_step(one(q), one(k), v, one(g), s1)
    assert torch.equal(o, gla.gla_step(*(one(t).contiguous() for t in (q, k)), v, one(g).contiguous(), s2))
    assert torch.equal(s1, s2)


def test_step_continues_a_chunked_forward():
    # a prompt of 2 chunks through the chunked forward, its ragged end and the answer through gla_step
    B, H, T, dk, dv, chunk = 2, 2, 139, 32, 64, 64
    d = inputs.generate(B, H, T, dk, dv, "bf16", 5)
    x = {n: t.cuda() for n, t in d.items()}
    cut = T // chunk * chunk
    head = {n: t[:, :, :cut].contiguous() for n, t in x.items()}
    f = gla.states_first_forward(head["q"], head["k"], head["v"], head["g"], chunk, 1, 1)
    state = f["h_final"]
    tail = {n: t[:, :, cut:] for n, t in x.items()}
    o1 = gla.gla_step(tail["q"][:, :, :7], tail["k"][:, :, :7], tail["v"][:, :, :7], tail["g"][:, :, :7], state)
    o = [f["o"], o1]
    for t in range(7, T - cut):
        o.append(gla.gla_step(*(tail[n][:, :, t:t + 1] for n in "qkvg"), state))
    got = torch.cat(o, 2).cpu().double().numpy()
    ref, last = oracle.gla_fwd(*(inputs.as_f64(d[n]) for n in "qkvg"))
    assert np.max(np.abs(got - ref)) <= 2e-2 * np.max(np.abs(ref))
    assert np.max(np.abs(state.cpu().double().numpy() - last)) <= 2e-2 * np.max(np.abs(last))


# ---------------------------------------------------------------------------------------- join

EPS = 1e-5


def join_reference(y, z, w_post, residual, scale, w_pre, act, d_out, d_normed):
    """Values and magnitudes (the same formulas over absolute values) in float64."""
    B, H, T, d = y.shape
    rows = lambda t: t.transpose(1, 2).reshape(B, T, H * d)  # noqa: E731
    heads = lambda t: t.reshape(B, T, H, d).transpose(1, 2)  # noqa: E731
    one = torch.ones((), dtype=torch.float64)
    ry = torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) if w_post is not None else one
    wo = w_post if w_post is not None else one
    yn = y * ry
    u = rows(yn * wo)
    if z is None:
        f, slope, slope_mag = one, one * 0, one * 0
    else:
        s = torch.sigmoid(z)
        f, slope = (z * s, s * (1 + z * (1 - s))) if act == "silu" else (s, s * (1 - s))
        slope_mag = s * (1 + z.abs() * (1 - s)) if act == "silu" else s
    sc = scale if scale is not None else one
    m = u * f
    out = m * sc + (residual if residual is not None else 0)
    out_mag = (m * sc).abs() + (residual.abs() if residual is not None else 0)
    r = {"out": (out, out_mag)}
    dO, dO_mag = (d_out, d_out.abs()) if d_out is not None else (0 * out, 0 * out)
    if w_pre is not None:
        rp = torch.rsqrt(out.square().mean(-1, keepdim=True) + EPS)
        n, n_mag = out * rp, out_mag * rp
        # the root's relative error is at most the mean of |out| out_mag over the mean of out^2
        root = (out_mag * out.abs()).mean(-1, keepdim=True) / (out.square().mean(-1, keepdim=True) + EPS)
        n_mag = n_mag + n.abs() * root
        r["normed"] = (n * w_pre, n_mag * w_pre.abs())
        if d_normed is not None:
            e = d_normed * w_pre
            dO = dO + rp * (e - n * (e * n).mean(-1, keepdim=True))
            dot = (e * n).abs().mean(-1, keepdim=True) + (e.abs() * n_mag).mean(-1, keepdim=True)
            dO_mag = dO_mag + (1 + root) * rp * (e.abs() + n_mag * dot + n.abs() * dot)
            r["dw_pre"] = ((d_normed * n).sum((0, 1)), (d_normed.abs() * n_mag).sum((0, 1)))
        else:
            r["dw_pre"] = (0 * w_pre, 0 * w_pre)
    if residual is not None:
        r["d_residual"] = (dO, dO_mag)
    if scale is not None:
        r["dscale"] = ((dO * m).sum((0, 1)), (dO_mag * m.abs()).sum((0, 1)))
    dm, dm_mag = dO * sc, dO_mag * sc.abs()
    if z is not None:
        r["dz"] = (dm * u * slope, dm_mag * u.abs() * slope_mag)
    du, du_mag = heads(dm * f), heads(dm_mag * f.abs())
    if w_post is not None:
        r["dw_post"] = ((du * yn).sum((0, 1, 2)), (du_mag * yn.abs()).sum((0, 1, 2)))
        e, e_mag = du * wo, du_mag * wo.abs()
        dy = ry * (e - yn * (e * yn).mean(-1, keepdim=True))
        dy_mag = ry * (e_mag + yn.abs() * (e_mag * yn.abs()).mean(-1, keepdim=True))
    else:
        dy, dy_mag = du, du_mag
    r["dy"] = (dy, dy_mag)
    return r


def join_inputs(seed, B, H, T, d, dt, st, post=True, gate=True, residual=True, scale=True, pre=True):
    gen = torch.Generator().manual_seed(seed)
    D = H * d
    a = dict(z=rnd(gen, B, T, D).mul(2).to(dt) if gate else None, w_post=(1 + rnd(gen, d) / 4).float() if post else None,
             residual=rnd(gen, B, T, D).to(st) if residual else None, scale=rnd(gen, D).float() if scale else None,
             w_pre=(1 + rnd(gen, D) / 4).float() if pre else None)
    return rnd(gen, B, H, T, d).to(dt), a, rnd(gen, B, T, D).to(st if residual else dt), rnd(gen, B, T, D).to(dt)


def check_join(y, a, d_out, d_normed, act, label, wrap=lambda t: t.cuda()):
    wide = lambda t: None if t is None else t.double()  # noqa: E731
    gpu = {n: None if t is None else (wrap(t) if t.dim() == 3 else t.cuda()) for n, t in a.items()}
    r = join_reference(wide(y), *(wide(a[n]) for n in ("z", "w_post", "residual", "scale", "w_pre")), act, wide(d_out),
                       wide(d_normed))
    yc = wrap(y)
    f = gla.gla_join_fwd(yc, act=act, eps=EPS, **gpu)
    b = gla.gla_join_bwd(yc, f, d_out=None if d_out is None else wrap(d_out),
                         d_normed=None if d_normed is None else wrap(d_normed), act=act, **gpu)
    torch.cuda.synchronize()
    res = dict(f, **b)
    k = 64 + (4 * float(a["z"].double().abs().max()) if a["z"] is not None else 0)
    chain = y.shape[0] * y.shape[2] // 512 + 32 + y.shape[1] * 130  # a lane's rows, a workgroup's, the partial sums'
    for n in ("out", "normed", "dy", "dz", "d_residual", "dw_post", "dscale", "dw_pre"):
        if n not in r:
            assert res[n] is None, n
            continue
        ref, mag = r[n]
        tol = (k + (chain if n in ("dw_post", "dscale", "dw_pre") else 0)) * U * mag
        h = half_step(res[n].dtype)
        inside(label + " " + n, res[n], ref, (tol + h * ref.abs()) * (1 + h))
    return f, b


JOIN_SIZES = [(1, 1, 1, 1), (2, 1, 3, 64), (1, 4, 5, 256), (2, 3, 33, 50), (1, 1, 7, 2048), (1, 16, 40, 128),
              (3, 2, 9, 7), (1, 2, 300, 129), (1, 1, 4, 8192), (2, 5, 6, 96), (1, 1, 3, 4099), (700, 1, 3, 16),
              (1, 3, 8, 520), (2, 1, 2, 1000), (1, 8, 11, 1024), (1, 15, 3, 520), (1, 126, 2, 65), (9, 1, 1, 1),
              (1, 1, 1100, 24)]


@pytest.mark.parametrize("dt,st", [(F32, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("B,H,T,d", JOIN_SIZES)
def test_join_against_the_formulas(B, H, T, d, dt, st):
    y, a, d_out, d_normed = join_inputs(B + T + d, B, H, T, d, dt, st)
    check_join(y, a, d_out, d_normed, "silu", "B%d H%d T%d d%d" % (B, H, T, d))


@pytest.mark.parametrize("left_out", [("post",), ("gate",), ("residual",), ("scale",), ("pre",), ("post", "gate"),
                                      ("residual", "pre", "scale"), ("post", "gate", "residual", "scale"),
                                      ("post", "gate", "residual", "scale", "pre")])
@pytest.mark.parametrize("d", [64, 33])
def test_join_parts(left_out, d):
    y, a, d_out, d_normed = join_inputs(4, 2, 3, 40, d, BF16, BF16, **{n: False for n in left_out})
    check_join(y, a, d_out, d_normed if a["w_pre"] is not None else None, "sigmoid", str(left_out))


@pytest.mark.parametrize("which", ["d_out", "d_normed"])
def test_join_one_gradient_alone(which):
    y, a, d_out, d_normed = join_inputs(6, 2, 2, 30, 64, F32, F32)
    check_join(y, a, d_out if which == "d_out" else None, d_normed if which == "d_normed" else None, "silu", which)


@pytest.mark.parametrize("off", [0, 1, 4, 8])
def test_join_views(off):
    # token-major y and slices of wider rows, at every alignment, bit for bit the contiguous result up to
    # the order of the sums (the slots are narrower where the alignment is)
    B, H, T, d = 2, 3, 21, 64
    y, a, d_out, d_normed = join_inputs(8, B, H, T, d, BF16, BF16)

    def wrap(t):
        rows = t.transpose(1, 2).reshape(B, T, H * d) if t.dim() == 4 else t
        wide = torch.full((B, T + 1, H * d + 2 * off + 8), math.nan, dtype=t.dtype, device="cuda")
        view = wide[:, 1:, off:off + H * d]
        view.copy_(rows)
        return view.unflatten(2, (H, d)).transpose(1, 2) if t.dim() == 4 else view

    check_join(y, a, d_out, d_normed, "silu", "off %d" % off, wrap)


def test_join_rows_of_zeros_and_large_rows():
    y, a, d_out, d_normed = join_inputs(9, 1, 2, 12, 32, F32, F32)
    y[:, :, 3] = 0
    y[:, 1, 4] *= 1e15
    a["residual"][:, 5] = 0
    y[:, :, 5] = 0
    check_join(y, a, d_out, d_normed, "silu", "zeros")


def test_join_in_the_residuals_place():
    y, a, _, _ = join_inputs(10, 2, 2, 50, 64, BF16, F32)
    gpu = {n: t.cuda() for n, t in a.items()}
    f = gla.gla_join_fwd(y.cuda(), eps=EPS, **gpu)
    r = gpu["residual"].clone()
    g = gla.gla_join_fwd(y.cuda(), eps=EPS, out=r, keep_rstd=False, **dict(gpu, residual=r))
    assert g["out"] is r and torch.equal(r, f["out"]) and torch.equal(g["normed"], f["normed"])
    assert g["rstd_post"] is None and g["rstd_pre"] is None
    with pytest.raises(ValueError, match="residual's place"):
        gla.gla_join_bwd(y.cuda(), g, d_out=r, **dict(gpu, residual=r))


def test_join_is_the_same_every_time():
    y, a, d_out, d_normed = join_inputs(13, 4, 4, 1000, 64, BF16, F32)
    gpu = {n: t.cuda() for n, t in a.items()}
    first = None
    for _ in range(4):
        f = gla.gla_join_fwd(y.cuda(), **gpu)
        b = gla.gla_join_bwd(y.cuda(), f, d_out=d_out.cuda(), d_normed=d_normed.cuda(), **gpu)
        first = first or b
        assert all(torch.equal(first[n], b[n]) for n in b)


# ------------------------------------------------------------------------------ used together

@pytest.mark.parametrize("order", ["zeco", "states_first"])
def test_chains_with_a_join_against_autograd(order):
    # gated linear attention, its output norm and gate, the residual and the next norm, forward and
    # backward through the method chains, against float64 autograd of the whole
    B, H, T, dk, dv, chunk, P = 1, 2, 128, 32, 64, 32, 2
    d = inputs.generate(B, H, T, dk, dv, "bf16", 3)
    _, a, d_out, d_normed = join_inputs(14, B, H, T, dv, BF16, F32)
    x = {n: t.cuda() for n, t in d.items()}
    join = dict({n: t.cuda() for n, t in a.items()}, act="silu", eps=EPS)
    if order == "zeco":
        f = gla.zeco_forward(x["q"], x["k"], x["v"], x["g"], chunk, P, 2, join=join)
        b = gla.zeco_backward(x["q"], x["k"], x["v"], x["g"], None, f, chunk, P, 2, join=join, d_out=d_out.cuda(),
                              d_normed=d_normed.cuda())
    else:
        f = gla.states_first_forward(x["q"], x["k"], x["v"], x["g"], chunk, P, 2, join=join)
        b = gla.states_first_backward(x["q"], x["k"], x["v"], x["g"], None, f, chunk, 2, join=join, d_out=d_out.cuda(),
                                      d_normed=d_normed.cuda())
    leaf = {n: t.double().requires_grad_() for n, t in dict(d, **a).items()}
    S, os = torch.zeros(B, H, dk, dv, dtype=torch.float64), []
    for t in range(T):
        S = torch.exp(leaf["g"][:, :, t])[..., None] * S + leaf["k"][:, :, t, :, None] * leaf["v"][:, :, t, None]
        os.append((leaf["q"][:, :, t, :, None] * S).sum(2))
    o = torch.stack(os, 2)
    u = o * torch.rsqrt(o.square().mean(-1, keepdim=True) + EPS) * leaf["w_post"]
    m = u.transpose(1, 2).reshape(B, T, H * dv) * torch.nn.functional.silu(leaf["z"])
    out = leaf["residual"] + leaf["scale"] * m
    normed = out * torch.rsqrt(out.square().mean(-1, keepdim=True) + EPS) * leaf["w_pre"]
    ((out * d_out.double()).sum() + (normed * d_normed.double()).sum()).backward()
    got = {"out": f["join"]["out"], "normed": f["join"]["normed"], **{n: b[n] for n in ("dq", "dk", "dv", "dg")},
           **{n: b["join"][n] for n in ("dz", "d_residual", "dw_post", "dscale", "dw_pre")}}
    ref = {"out": out, "normed": normed, "dq": leaf["q"].grad, "dk": leaf["k"].grad, "dv": leaf["v"].grad,
           "dg": leaf["g"].grad, "dz": leaf["z"].grad, "d_residual": leaf["residual"].grad,
           "dw_post": leaf["w_post"].grad, "dscale": leaf["scale"].grad, "dw_pre": leaf["w_pre"].grad}
    for n, t in got.items():
        r = ref[n].detach()
        # the chunked operator's own tolerance in bf16 (2e-2 of the largest value) on o passes through the
        # norm's 1 / rms, largest where a head's o is smallest, to everything behind it
        err = float((t.cpu().double() - r).norm() / r.norm())
        assert err <= 4e-2, (n, err)


def test_a_recurrent_block_as_it_is_used():
    # two layers' worth: norm -> recurrence -> gate and residual -> norm -> recurrence, with a padded batch
    B, T, D = 3, 200, 64
    gen = torch.Generator().manual_seed(21)
    x = rnd(gen, B, T, D).float()
    z, w = rnd(gen, B, T, D).float(), (1 + rnd(gen, D) / 8).float()
    g = (torch.nn.functional.logsigmoid(rnd(gen, B, T, D)) / 4).float()
    lens = torch.tensor([200, 0, 77])
    xc, zc, wc, gc, ln = x.cuda(), z.cuda(), w.cuda(), g.cuda(), lens.to(torch.int32).cuda()
    f0 = gla.gla_join_fwd(xc[:, None], w_pre=wc, eps=EPS)
    h1, _, _ = gla.gla_recur_fwd(f0["normed"], gc, lens=ln, mode="norm")
    f1 = gla.gla_join_fwd(h1[:, None], z=zc, residual=xc, w_pre=wc, eps=EPS)
    h2, _, _ = gla.gla_recur_fwd(f1["normed"], gc, lens=ln, mode="norm")
    norm = lambda t: t * torch.rsqrt(t.square().mean(-1, keepdim=True) + EPS) * w.double()  # noqa: E731
    zero = torch.zeros(B, D, dtype=torch.float64)
    a1 = recur_reference(norm(x.double()), g.double(), zero, lens, "norm")["h"][0]
    out = x.double() + a1 * torch.nn.functional.silu(z.double())
    a2 = recur_reference(norm(out), g.double(), zero, lens, "norm")["h"][0]
    assert float((h2.cpu().double() - a2).abs().max()) <= 1e-4
    assert float((f1["out"].cpu().double() - out).abs().max()) <= 1e-4


def test_a_served_block_prompt_then_tokens():
    # a prompt through the chunked chain with its join, then token by token: gla_step on the prompt's final
    # state, and the join in the residual's place, against float64 of the whole sequence
    B, H, T, dk, dv, chunk, more = 2, 2, 128, 32, 64, 32, 5
    d = inputs.generate(B, H, T + more, dk, dv, "bf16", 9)
    _, a, _, _ = join_inputs(15, B, H, T + more, dv, BF16, F32)
    x = {n: t.cuda() for n, t in d.items()}
    rows = {n: t.cuda() for n, t in a.items() if n in ("z", "residual")}
    w = {n: t.cuda() for n, t in a.items() if n not in rows}
    part = lambda n, lo, hi: x[n][:, :, lo:hi].contiguous()  # noqa: E731
    f = gla.states_first_forward(*(part(n, 0, T) for n in "qkvg"), chunk, 1, 1,
                                 join=dict(w, z=rows["z"][:, :T], residual=rows["residual"][:, :T], eps=EPS))
    state, outs = f["h_final"], [f["join"]]
    for t in range(T, T + more):
        o = gla.gla_step(*(x[n][:, :, t:t + 1] for n in "qkvg"), state)
        r = rows["residual"][:, t:t + 1].contiguous()
        outs.append(gla.gla_join_fwd(o, z=rows["z"][:, t:t + 1], residual=r, out=r, eps=EPS, keep_rstd=False, **w))
    o, _ = oracle.gla_fwd(*(inputs.as_f64(d[n]) for n in "qkvg"))
    ref = join_reference(torch.from_numpy(o), *(a[n].double() for n in ("z", "w_post", "residual", "scale", "w_pre")),
                         "silu", None, None)
    for n in ("out", "normed"):
        got = torch.cat([j[n] for j in outs], 1).cpu().double()
        assert float((got - ref[n][0]).norm() / ref[n][0].norm()) <= 4e-2, n
        tail = got[:, T:] - ref[n][0][:, T:]
        assert float(tail.norm() / ref[n][0][:, T:].norm()) <= 4e-2, n


def test_two_calls_at_once():
    # scans of several tiles on two streams, each with a workspace of its own
    x, g, dh, h0, dhT = (t.cuda() for t in recur_inputs(41, 1, 30000, 320, BF16, "weak"))
    want = gla.gla_recur_fwd(x, g, h0=h0, mode="norm")
    wantb = gla.gla_recur_bwd(x, g, dh, want[1], dhT=dhT, mode="norm")
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for i in range(6):
        with torch.cuda.stream(streams[i % 3]):
            f = gla.gla_recur_fwd(x, g, h0=h0, mode="norm")
            got.append(f + gla.gla_recur_bwd(x, g, dh, f[1], dhT=dhT, mode="norm"))
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(s, t) for s, t in zip(r, want + wantb))


def test_other_streams_and_replayed_graphs():
    # every operator on a side stream, then captured once and replayed three times on new inputs with eager
    # work between, each replay against the eager result bit for bit
    B, T, D, H, d = 2, 300, 64, 2, 32
    xr, g, dh, h0, dhT = (t.cuda() for t in recur_inputs(31, B, T, D, BF16))
    y, a, d_out, d_normed = join_inputs(32, B, H, T, d, BF16, BF16)
    y, d_out, d_normed, a = y.cuda(), d_out.cuda(), d_normed.cuda(), {n: t.cuda() for n, t in a.items()}
    q, k, v, gs, pool = (t.cuda() for t in step_inputs(33, B, H, 1, 32, 48, BF16))
    state = pool.clone()

    def work():
        h, c, hf = gla.gla_recur_fwd(xr, g, h0=h0, mode="norm")
        b = gla.gla_recur_bwd(xr, g, dh, c, dhT=dhT, mode="norm")
        f = gla.gla_join_fwd(y, **a)
        jb = gla.gla_join_bwd(y, f, d_out=d_out, d_normed=d_normed, **a)
        state.copy_(pool)
        o = gla.gla_step(q, k, v, gs, state)
        return [h, c, hf, *b, f["out"], f["normed"], *(jb[n] for n in sorted(jb)), o, state]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = [t.clone() for t in work()]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(s, t) for s, t in zip(first, work()))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        static = work()
    gen = torch.Generator("cuda").manual_seed(1)
    for _ in range(3):
        for t in (xr, dh, y, d_out, q, k):
            t.copy_(torch.randn(t.shape, device="cuda", generator=gen))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in static]
        assert all(torch.equal(s, t) for s, t in zip(got, work()))
        torch.cuda.synchronize()


def test_offsets_past_32_bits():
    # a sequence of more than 2^32 elements: its end against the same tokens run on their own
    T, D = 4_200_000, 1024
    x = torch.zeros(1, T, D, dtype=BF16, device="cuda")
    g = torch.full((1, 1, D), -0.01, device="cuda").expand(1, T, D)
    tail = torch.randn(1, 500, D, device="cuda").to(BF16)
    x[:, -500:] = tail
    h, _, last = gla.gla_recur_fwd(x, g, keep_chunk_states=False)
    ref, _, want = gla.gla_recur_fwd(tail, g[:, :500])
    # the two runs' chunks lie apart by part of a chunk, so the same terms are combined in other groups:
    # each is within U (8 H + W) of the recurrence, H its sum of absolute terms, and with one decay a for
    # all tokens W_t = a (W_{t-1} + 5.02 H_{t-1}) stays below 5.02 H_max / (1 - a) (H_max the largest H)
    H = gla.gla_recur_fwd(tail.float().abs(), g[:, :500])[0].amax(1).double()
    tol = 2 * U * (8 + 5.02 / (1 - math.exp(-0.01))) * H
    assert ((last.double() - want.double()).abs() <= tol).all()
    step = half_step(BF16)
    diff = (h[:, -500:].double() - ref.double()).abs()
    assert (diff <= tol[:, None] + 2 * step * (ref.double().abs() + tol[:, None])).all()
    assert not h[:, :-500].any()


@pytest.mark.parametrize("dt,st", [(F32, F32), (BF16, F32)])
@pytest.mark.parametrize("B,H,T,d", [(1, 2048, 2, 4), (1, 2048, 3, 3), (2, 2047, 2, 1), (1, 1100, 2, 2)])
def test_join_with_many_narrow_heads(B, H, T, d, dt, st):
    y, a, d_out, d_normed = join_inputs(B + T + d, B, H, T, d, dt, st)
    check_join(y, a, d_out, d_normed, "silu", "B%d H%d T%d d%d" % (B, H, T, d))


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("dk,dv", [(48, 32), (100, 17), (1, 5), (17, 64), (192, 8), (64, 32)])
def test_step_with_a_value_that_is_not_finite(dk, dv, dt, bad):
    # one column of v at token 0 is not finite; a reset at token 1 drops it.  k and q are positive, so
    # that the sums over the rows are infinite, not NaN, where the formula says so
    B, H, n = 2, 2, 4
    q, k, v, g, pool = step_inputs(dk, B, H, n, dk, dv, dt)
    q, k = q.abs() + 0.5, k.abs() + 0.5
    v[:, :, 0, 0] = bad
    g[:, :, 1] = -math.inf
    state = pool.cuda()
    o = gla.gla_step(q.cuda(), k.cuda(), v.cuda(), g.cuda(), state).cpu().double()
    first = o[:, :, 0, 0]
    assert (torch.isnan(first) if math.isnan(bad) else first == bad).all()
    v[:, :, 0, 0] = 0
    ref, tol, S, tolS = step_reference(q.double(), k.double(), v.double(), g.double(), pool[:B].double())
    o[:, :, 0, 0] = ref[:, :, 0, 0]
    inside("o", o, ref, (tol + half_step(dt) * ref.abs()) * (1 + half_step(dt)))
    inside("state", state[:B], S, tolS + U * S.abs())


def test_outputs_in_a_views_gaps_and_next_to_inputs():
    # out between two of y's sequences; x, g and h side by side.  Nothing overlaps, and the results are those of
    # separate tensors; one element further it does
    B, H, T, d = 3, 2, 20, 32
    y, a, _, _ = join_inputs(3, B, H, T, d, BF16, BF16)
    gpu = {n: t.cuda() for n, t in a.items()}
    want = gla.gla_join_fwd(y.cuda(), eps=EPS, **gpu)
    n = B * H * T * d
    flat = torch.zeros(4 * n, dtype=BF16, device="cuda")
    view = flat[:3 * n].view(B, n)[:, :n // B].view(B, H, T, d)
    view.copy_(y)
    one = gla.gla_join_fwd(view[::2], eps=EPS, out=flat[n:n + 2 * n // 3].view(2, T, H * d),
                           **{k: t if t.dim() == 1 else t[::2] for k, t in gpu.items()})
    assert torch.equal(one["out"], want["out"][::2]) and torch.equal(one["normed"], want["normed"][::2])
    x, g, _, _, _ = recur_inputs(4, 2, 70, 64, F32)
    want, _, last = gla.gla_recur_fwd(x.cuda(), g.cuda())
    m = x.numel()
    both = torch.zeros(3 * m, device="cuda")
    both[:m], both[m:2 * m] = x.cuda().flatten(), g.cuda().flatten()
    h, _, f = gla.gla_recur_fwd(both[:m].view(2, 70, 64), both[m:2 * m].view(2, 70, 64), h=both[2 * m:].view(2, 70, 64))
    assert torch.equal(h, want) and torch.equal(f, last)
    for lo in (2 * m - 1, m - 4):
        with pytest.raises(gla.GLAError, match="must not overlap"):
            gla.gla_recur_fwd(both[:m].view(2, 70, 64), both[m:2 * m].view(2, 70, 64), h=both[lo:lo + m].view(2, 70, 64))


@pytest.mark.parametrize("B", [1, 2])
def test_an_output_between_a_views_rows(B):
    # x is every other block of `wide`; h takes a whole block between
    T, D = 3, 16
    wide = torch.zeros(2 * B, B * T, D, device="cuda")
    x = wide[::2][:, :T]
    x.copy_(torch.randn(B, T, D))
    g = -torch.rand(B, T, D, device="cuda")
    want = gla.gla_recur_fwd(x.clone(), g)[0]
    h = wide[1].view(B, T, D)
    assert torch.equal(gla.gla_recur_fwd(x, g, h=h)[0], want) and torch.equal(wide[1].view(B, T, D), want)
    if B > 1:
        over = wide.view(-1)[B * T * D + D:][:B * T * D].view(B, T, D)  # ends in the next block's first row
        with pytest.raises(gla.GLAError, match="must not overlap"):
            gla.gla_recur_fwd(x, g, h=over)


def test_join_with_the_longest_sequences():
    # T = 2^31 - 1: a row's step passes 2^31 at the first sequence's end.  With every part left out out is y
    # and dy is d_out
    B, T = 2, 2 ** 31 - 1
    y = torch.empty(B, 1, T, 1, dtype=BF16, device="cuda")
    y.view(torch.int16).view(-1)[:] = 0
    ends = torch.randn(2, 1 << 20, device="cuda").to(BF16)  # around the sequences' border and at the far end
    flat = y.view(-1)
    flat[T - (1 << 19):T + (1 << 19)] = ends[0]
    flat[-(1 << 20):] = ends[1]
    f = gla.gla_join_fwd(y)
    out = f["out"].view(-1)
    step = 1 << 28
    assert all(torch.equal(out[i:i + step], flat[i:i + step]) for i in range(0, flat.numel(), step))
    dy = gla.gla_join_bwd(y, f, d_out=y.view(B, T, 1))["dy"].view(-1)
    assert all(torch.equal(dy[i:i + step], flat[i:i + step]) for i in range(0, flat.numel(), step))


def test_step_fills_the_longest_call():
    # a row that is left out, n = 2^31 - 1 tokens of one value: zeros up to the last, nothing behind
    n = 2 ** 31 - 1
    one = torch.ones(1, 1, 1, 1, dtype=BF16, device="cuda").expand(1, 1, n, 1)
    g = torch.zeros(1, 1, 1, 1, device="cuda").expand(1, 1, n, 1)
    whole = torch.ones(n + 1025, dtype=BF16, device="cuda")
    o = whole[1024:-1].view(1, 1, n, 1)
    gla.gla_step(one, one, one, g, torch.zeros(1, 1, 1, 1, device="cuda"),
                 slots=torch.tensor([-1], dtype=torch.int32, device="cuda"), o=o)
    step = 1 << 28
    assert not any(whole[i:min(i + step, 1024 + n)].any() for i in range(1024, 1024 + n, step))
    assert (whole[:1024] == 1).all() and whole[-1] == 1


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("T", [10, 120, 700])
def test_recur_plain_gate_gradient_does_not_read_the_input(T, dt, bad):
    # beta = 1: dg_t = a_t h_{t-1} G_t whatever x_t is.  The token after is a reset, so nothing else has it
    x, g, dh, h0, dhT = (t.cuda() for t in recur_inputs(T, 2, T, 40, dt))
    at = [1, T // 2, T - 3]
    g[:, [i + 1 for i in at]] = -math.inf
    x[:, at] = 0
    h, c, last = gla.gla_recur_fwd(x, g, h0=h0)
    want = gla.gla_recur_bwd(x, g, dh, c, dhT=dhT)
    y = x.clone()
    y[:, at] = bad
    h1, c1, last1 = gla.gla_recur_fwd(y, g, h0=h0)
    assert torch.equal(c1, c) and torch.equal(last1, last)
    assert (torch.isnan(h1[:, at]) if math.isnan(bad) else h1[:, at] == bad).all()
    for s, t in zip(gla.gla_recur_bwd(y, g, dh, c1, dhT=dhT), want):
        assert torch.isfinite(t).all() and torch.equal(s, t)


def test_strides_of_dimensions_that_are_not_there():
    # through the C calls: h of a [B][T][D] tensor, h and t of a [B][D] one may hold anything, and the token
    # stride of a single token in the residual's place is not looked at
    import ctypes
    lib = gla.load_library()
    st = lambda b, h, t: (ctypes.c_longlong * 3)(b, h, t)  # noqa: E731
    stream = torch.cuda.current_stream().cuda_stream
    B, T, D = 2, 5, 16
    x, g, _, _, _ = (t.cuda() for t in recur_inputs(1, B, T, D, F32))
    want, h = gla.gla_recur_fwd(x, g)[0], torch.empty_like(x)
    s = st(T * D, -7, D)
    assert lib.gla_recur_fwd(x.data_ptr(), s, g.data_ptr(), s, None, None, h.data_ptr(), None, None, B, T, D, 0, 0, None,
                             0, stream) == 0
    assert torch.equal(h, want)
    one, s = torch.empty(B, D, device="cuda"), st(T * D, -1, -(1 << 40))
    states = [torch.zeros(B, D, device="cuda") for _ in range(2)]
    assert lib.gla_recur_step(x.data_ptr(), s, g.data_ptr(), s, states[0].data_ptr(), None, one.data_ptr(), B, D, B, 0, 0,
                              stream) == 0
    assert torch.equal(one, gla.gla_recur_step(x[:, 0], g[:, 0], states[1])) and torch.equal(*states)
    y, r = torch.randn(B, 1, 1, D, device="cuda"), torch.randn(B, 1, D, device="cuda")
    want = gla.gla_join_fwd(y, residual=r)["out"]
    assert lib.gla_join_fwd(y.data_ptr(), None, None, None, None, r.data_ptr(), st(D, -1, 999), None, None, r.data_ptr(),
                            None, None, None, B, 1, 1, D, 0, 1e-6, 0, 0, stream) == 0
    assert torch.equal(r, want)


@pytest.mark.parametrize("d", [64, 51])
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("off", [1, 3, 4, 8])
def test_join_views_bit_for_bit(off, dt, d):
    # a row's slots and sums do not depend on where it lies, so views give the contiguous tensors' bits
    B, H, T = 2, 3, 21
    y, a, d_out, d_normed = join_inputs(8, B, H, T, d, dt, dt)

    def cut(t):
        rows = t.transpose(1, 2).reshape(B, T, H * d) if t.dim() == 4 else t
        wide = torch.full((B, T + 1, H * d + 2 * off + 8), math.nan, dtype=t.dtype, device="cuda")
        view = wide[:, 1:, off:off + H * d]
        view.copy_(rows)
        return view.unflatten(2, (H, d)).transpose(1, 2) if t.dim() == 4 else view

    res = []
    for wrap in (cut, lambda t: t.cuda()):
        gpu = {n: wrap(t) if t.dim() == 3 else t.cuda() for n, t in a.items()}
        f = gla.gla_join_fwd(wrap(y), **gpu)
        b = gla.gla_join_bwd(wrap(y), f, d_out=wrap(d_out), d_normed=wrap(d_normed), **gpu)
        res.append({**f, **b})
    assert all(torch.equal(t, res[1][n]) for n, t in res[0].items())
