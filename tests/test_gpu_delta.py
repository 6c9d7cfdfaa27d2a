"""The gated delta rule (gla_delta_*) and layer norm (gla_layernorm_*) against plain float64 code written from their
definitions: the rule token by token, forward and adjoint.

Tolerances.  A rounding to nearest with a half step of h is off by at most h of the value, in the mean square by
h / sqrt(3) of it at most; roundings are independent of each other, so n of them on the way to a result leave
sqrt(n) h / sqrt(3) in the 2-norm, relative to the terms that are summed, in the root of their squares' sum (the result
itself where that is more: terms of one sign).  Terms may cancel: with one channel, dk = beta D e - A de can be -0.0079 =
-0.0369 + 0.0076 + 0.0214, and two roundings of 2^-8 of the first of them alone are 2.9e-4.  The squares of N such errors
add up to N times their mean and, at four standard deviations, 4 sqrt(2 N) more, a factor of sqrt(1 + 5.7 / sqrt(N)) in the
norm.  The terms of a state are the one that enters the chunk, decayed, and the chunk's writes, each rounded by itself:
with few channels the writes replace the state again and again, and S^2 is less than the sum of their squares (18 heads of
288 tokens, 4 x 80, bf16, weak gates: dq's norm is 827, its terms' 828 by S and 2386 by what S is summed from, so that four
roundings of 2^-8 / sqrt(3) may leave up to 1.3e-2 of dq; they leave 4.8e-3).
Likewise the gradient of a state (9 heads of 733 tokens, 1 x 64: dh0's norm is 16, its terms' 222).
  - bf16 results, h = 2^-8: o of a training step n = 1; of a forward-only call, where the state, W, P and o are rounded,
    n = 4; dv 1; dq (state or W, H, dq) and dk (the same with one more) 4.
  - float32 results beside bf16 inputs: two bf16 parts a factor, h = 2^-17: the state passes four split factors and
    two products without the low parts' product, n = 6; the backward as many more, n = 12.
  - float32 inputs: sums of up to 128 and 64 terms, one after the other, h = 2^-24 each, so n = 192 a product, and as
    many products as above.
A single element may be off by 8 times that, relative to its head's mean square or itself.
"""
import math

import pytest
import torch

from sequence_state_scan_amd import gla

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
STAGES = {"o": 6, "h_final": 6, "dq": 12, "dk": 12, "dv": 12, "dbeta": 12, "dh0": 12, "dg": 12}
ROUNDED = {"o": 1, "o only": 4, "dq": 4, "dk": 4, "dv": 1}


def share(name, dt, out_dt):
    """The relative error in the 2-norm that a result may have."""
    if dt == F32:
        return math.sqrt(192 * STAGES[name.split()[0]] / 3) * 2.0 ** -24
    fine = math.sqrt(STAGES[name.split()[0]] / 3) * 2.0 ** -17
    return fine if out_dt == F32 else fine + math.sqrt(ROUNDED[name] / 3) * 2.0 ** -8


def near(label, got, ref, tol, terms=None):
    """got within tol of ref ([B, heads, ...]); terms: the root of the summed terms' squares."""
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, (label, got.shape, ref.shape)
    assert torch.isfinite(got).all(), "%s: not finite" % label
    size = ref.abs() if terms is None else torch.hypot(ref, terms)
    tol = tol * math.sqrt(1 + 5.7 / math.sqrt(max(1, ref.numel())))
    off, norm = float((got - ref).norm()), float(size.norm())
    assert off <= tol * norm + 1e-30, "%s: off by %.3g of its terms where %.3g is allowed" % (label, off / max(norm, 1e-300), tol)
    head = size.flatten(2).square().mean(-1).sqrt().reshape(ref.shape[:2] + (1,) * (ref.dim() - 2))
    worst = ((got - ref).abs() - 8 * tol * (size + head)).max() if ref.numel() else torch.zeros(())
    assert float(worst) <= 1e-30, "%s: one element off by %.3g more than allowed" % (label, float(worst))


def unit(t):
    return t / (t.square().sum(-1, keepdim=True) + 1e-6).sqrt()


def inputs(seed, B, H, Hk, T, dk, dv, dt, gates="mid", resets=0):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    x = {"q": unit(rnd(B, Hk, T, dk)).to(dt), "k": unit(rnd(B, Hk, T, dk)).to(dt), "v": rnd(B, H, T, dv).to(dt)}
    pre = rnd(B, H, T)
    x["g"] = {"mid": torch.nn.functional.logsigmoid(pre) / 8, "weak": -pre.abs() / 1024, "strong": -6 * pre.abs(),
              "zero": 0 * pre, "mixed": -pre.abs() * torch.where(rnd(B, H, T) > 1, 40.0, 0.02)}[gates].float()
    if resets:
        x["g"][:, :, torch.randint(0, T, (resets,), generator=gen)] = -math.inf
    x["beta"] = torch.sigmoid(rnd(B, H, T)).float()
    x["do"], x["h0"], x["dhT"] = rnd(B, H, T, dv).to(dt), (0.3 * rnd(B, H, dk, dv)).float(), (0.3 * rnd(B, H, dk, dv)).float()
    return x


def reference(x, lens=None):
    """The rule and its adjoint, token by token."""
    q, k, v, g, beta, do = (x[n].double() for n in ("q", "k", "v", "g", "beta", "do"))
    B, Hk, T, dk = q.shape
    H, dv = v.shape[1], v.shape[3]
    G = H // Hk
    q, k = q.repeat_interleave(G, 1), k.repeat_interleave(G, 1)
    S = torch.zeros(B, H, dk, dv, dtype=torch.float64) if x.get("h0") is None else x["h0"].double()
    a = g.exp()
    lens = torch.full((B,), T) if lens is None else lens.clamp(0, T)
    live = torch.arange(T)[None, :] < lens[:, None]
    q, k, v, do = (torch.where(live[:, None, :, None], t, 0.0) for t in (q, k, v, do))
    a, beta = torch.where(live[:, None], a, 1.0), torch.where(live[:, None], beta, 0.0)
    o, kept = torch.zeros_like(v), []
    size = {}  # of the terms
    size["o"], size["dq"] = torch.zeros_like(v), torch.zeros_like(q)
    root = lambda t, *dims: t.square().sum(dims).sqrt()  # noqa: E731
    for t in range(T):
        if t % 64 == 0:
            parts = S.square()  # of the state that enters the chunk and of the chunk's writes
        A = a[:, :, t, None, None] * S
        e = v[:, :, t] - (k[:, :, t, :, None] * A).sum(2)
        write = (beta[:, :, t, None] * k[:, :, t])[..., None] * e[:, :, None]
        parts = a[:, :, t, None, None].square() * parts
        kept.append((S, A, e, parts))
        parts = parts + write.square()
        S = A + write
        o[:, :, t] = (q[:, :, t, :, None] * S).sum(2)
        size["o"][:, :, t] = (q[:, :, t, :, None].square() * parts).sum(2).sqrt()
        size["dq"][:, :, t] = (do[:, :, t, None, :].square() * parts).sum(-1).sqrt()
    size["h_final"], size["last token"] = parts.sqrt(), torch.hypot(A, S - A)
    r = {"o": o, "h_final": S}
    D = torch.zeros_like(S) if x.get("dhT") is None else x["dhT"].double()
    dq, dkey, dval, dg, db = (torch.zeros_like(t) for t in (q, k, v, a, beta))
    at, ends = torch.zeros_like(a), {}
    size.update(dk=torch.zeros_like(k), dv=torch.zeros_like(v), dbeta=torch.zeros_like(a))
    for t in range(T - 1, -1, -1):
        before, A, e, parts = kept[t]
        if t % 64 == 63 or t == T - 1:
            back = D.square()  # of the gradient, as parts
        if t % 256 == 255 or t == T - 1:
            ends[t] = (S.flatten(2).norm(dim=-1) * D.flatten(2).norm(dim=-1))
        dq[:, :, t] = (S * do[:, :, t, None, :]).sum(-1)
        was, D = D, D + q[:, :, t, :, None] * do[:, :, t, None, :]
        De = (D * e[:, :, None, :]).sum(-1)
        db[:, :, t] = (k[:, :, t] * De).sum(-1)
        de = beta[:, :, t, None] * (k[:, :, t, :, None] * D).sum(2)
        dval[:, :, t] = de
        dkey[:, :, t] = beta[:, :, t, None] * De - (A * de[:, :, None, :]).sum(-1)
        D = D - k[:, :, t, :, None] * de[:, :, None, :]
        back = back + (q[:, :, t, :, None] * do[:, :, t, None, :]).square() + (k[:, :, t, :, None] * de[:, :, None, :]).square()
        b = beta[:, :, t, None]
        own = (q[:, :, t, :, None] * do[:, :, t, None, :] * e[:, :, None]).sum(-1)  # of the token's own output
        size["dk"][:, :, t] = torch.stack([b * root(was * e[:, :, None], -1), b * own, (parts * de[:, :, None].square()).sum(-1).sqrt()]).square().sum(0).sqrt()
        size["dv"][:, :, t] = b * torch.hypot(root(k[:, :, t, :, None] * was, 2), (k[:, :, t] * q[:, :, t]).sum(-1, keepdim=True) * do[:, :, t])
        size["dbeta"][:, :, t] = torch.hypot(root(k[:, :, t, :, None] * was * e[:, :, None], -1, -2), root(k[:, :, t] * own, -1))
        dg[:, :, t] = (D * before).sum((-1, -2)) * a[:, :, t]
        at[:, :, t] = o[:, :, t].norm(dim=-1) * do[:, :, t].norm(dim=-1) + v[:, :, t].norm(dim=-1) * de.norm(dim=-1)
        D, back = a[:, :, t, None, None] * D, a[:, :, t, None, None].square() * back
        S = before
    # the size of dg's terms: those of the tokens up to the next 256th, and <S, D> there
    terms, run = torch.zeros_like(at), None
    for t in range(T - 1, -1, -1):
        run = ends[t].square() if t in ends else run
        run = run + at[:, :, t].square()
        terms[:, :, t] = run.sqrt()
    zero = lambda t: torch.where(live[:, None], t, 0.0)  # noqa: E731
    heads = lambda t: t.unflatten(1, (Hk, G)).sum(2)  # noqa: E731
    size.update(dq=heads(size["dq"].square()).sqrt(), dk=heads(size["dk"].square()).sqrt(), dh0=back.sqrt(), dg=terms)
    r.update(dq=heads(dq), dk=heads(dkey), dv=dval, dg=zero(dg), dbeta=zero(db), dh0=D, size=size)
    return r


def on_gpu(x):
    return {n: None if t is None else t.cuda() for n, t in x.items()}


def call(c, lens=None, **kw):
    a = tuple(c[n] for n in ("q", "k", "v", "g", "beta"))
    o, h_final, saved = gla.gla_delta_fwd(*a, h0=c.get("h0"), lens=lens, **kw)
    grads = gla.gla_delta_bwd(*a, o, c["do"], saved, lens=lens, dhT=c.get("dhT"))
    return dict(zip(("o", "h_final", "dq", "dk", "dv", "dg", "dbeta", "dh0"), (o, h_final) + grads))


def check(x, lens=None, label="", wrap=on_gpu):
    dt = x["q"].dtype
    r = reference(x, lens)
    ln = None if lens is None else lens.to(torch.int32).cuda()
    c = wrap(x)
    got = call(c, ln)
    only = gla.gla_delta_fwd(*(c[n] for n in ("q", "k", "v", "g", "beta")), h0=c.get("h0"), lens=ln, keep_saved=False)
    assert only[2] is None
    torch.cuda.synchronize()
    for n, t in got.items():
        near("%s %s" % (label, n), t, r[n], share(n, dt, t.dtype), r["size"][n])
    near(label + " o only", only[0], r["o"], share("o only", dt, dt), r["size"]["o"])
    near(label + " h_final only", only[1], r["h_final"], share("h_final", dt, F32), r["size"]["h_final"])
    return got


SIZES = [(1, 1, 1, 1, 1, 1), (2, 2, 1, 7, 3, 5), (1, 3, 3, 63, 16, 20), (1, 2, 2, 64, 32, 64), (2, 1, 1, 65, 33, 65),
         (1, 2, 1, 200, 100, 80), (2, 4, 2, 333, 48, 80), (1, 1, 1, 700, 128, 130), (1, 6, 2, 130, 128, 128)]


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("B,H,Hk,T,dk,dv", SIZES)
def test_delta_against_the_rule(B, H, Hk, T, dk, dv, dt):
    x = inputs(T + dk, B, H, Hk, T, dk, dv, dt)
    check(x, label="B%d H%d/%d T%d %dx%d" % (B, H, Hk, T, dk, dv))


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("gates", ["weak", "strong", "zero", "mixed"])
def test_delta_gates(gates, dt):
    check(inputs(7, 1, 2, 2, 300, 64, 48, dt, gates), label=gates)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("T,dk,dv", [(1100, 64, 64), (2500, 32, 200), (1601, 100, 80)])
def test_delta_segments(T, dk, dv, dt):
    # long enough for the sequence to be cut into segments that run side by side
    x = inputs(T, 2, 1, 1, T, dk, dv, dt, gates="weak")
    check(x, label="segments")
    check(x, lens=torch.tensor([T - 517, 400]), label="segments, lens")


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("T,dk,dv", [(40, 16, 16), (4400, 16, 16), (700, 128, 100)])
def test_delta_first_gate(T, dk, dv, dt):
    # the first gate scales h0, so its gradient is <h0, dh0> whatever the tokens after it add up to: sums of dk / 4 products a
    # lane, six exchanges, a number per 16 columns, and four roundings of the result
    c = on_gpu(inputs(T, 2, 2, 2, T, dk, dv, dt))
    got = call(c)
    terms = c["h0"].double() * got["dh0"].double()
    steps = max(32, 1 << (dk - 1).bit_length()) / 4 + 6 + math.ceil(dv / 16) + 4
    off = (got["dg"][:, :, 0].double() - terms.sum((-1, -2))).abs()
    assert bool((off <= steps * 2.0 ** -24 * terms.abs().sum((-1, -2))).all())


def test_delta_without_the_optional_tensors():
    x = inputs(5, 2, 2, 2, 150, 40, 30, F32)
    x["h0"] = x["dhT"] = None
    check(x, label="no states")


@pytest.mark.parametrize("dt", [F32, BF16])
def test_delta_lengths_and_what_stands_behind_them(dt):
    # lengths of zero and one, at a chunk's end and past it, a full one, values outside 0..T; NaN behind the ends
    T = 333
    lens = torch.tensor([0, 1, T, 64, 65, 200, -3, T + 9])
    x = inputs(3, len(lens), 2, 1, T, 32, 40, dt)
    clean = check(x, lens, "lens")
    for b, n in enumerate(lens.clamp(0, T).tolist()):
        for name in ("q", "k", "v", "do"):
            x[name][b, :, n:] = math.nan
        x["g"][b, :, n:], x["beta"][b, :, n:] = math.inf, math.nan
    dirty = call(on_gpu(x), lens.to(torch.int32).cuda())
    for n in clean:
        assert torch.equal(clean[n], dirty[n]), n


def test_delta_resets_cut_documents_apart():
    x = inputs(11, 1, 2, 2, 400, 48, 40, F32, resets=5)
    check(x, label="resets")
    cut = 201
    x["g"][:, :, cut] = -math.inf
    a = call(on_gpu(x))
    x["v"][:, :, :cut] *= 3
    x["h0"] *= -2
    b = call(on_gpu(x))
    # what stands before a reset changes nothing behind it (the same tokens of a chunk are the same numbers), and a
    # reset's own gate has no slope
    near("behind a reset", b["o"][:, :, cut:], a["o"][:, :, cut:].cpu().double(), share("o", F32, F32))
    assert torch.equal(a["dg"][:, :, cut], torch.zeros_like(a["dg"][:, :, cut]))


@pytest.mark.parametrize("dt", [F32, BF16])
def test_delta_betas(dt):
    # tokens that write nothing (their gradient is what writing would do), and a beta of up to 2
    x = inputs(13, 1, 2, 1, 170, 64, 32, dt)
    x["beta"][:, :, ::3] = 0
    x["beta"][:, 0] *= 2
    got = check(x, label="betas")
    assert float(got["dbeta"][:, :, ::3].abs().max()) > 0.01


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("off,pad", [(0, 8), (3, 5), (8, 0), (1, 0)])
def test_delta_views(dt, off, pad):
    # [B, T, heads, d] slices of wider rows at every alignment, gates with heads last, an expanded batch
    B, H, Hk, T, dk, dv = 2, 4, 2, 150, 64, 40

    def wrap(x):
        def rows(t):
            n, d = t.shape[1], t.shape[3]
            wide = torch.full((B, T + 2, off + n * d + pad), math.nan, dtype=t.dtype, device="cuda")
            v = wide[:, 1:T + 1, off:off + n * d].unflatten(-1, (n, d)).transpose(1, 2)
            v.copy_(t)
            return v
        c = on_gpu(x)
        for n in ("q", "k", "v", "do"):
            c[n] = rows(x[n])
        for n in ("g", "beta"):
            c[n] = x[n].cuda().transpose(1, 2).contiguous().transpose(1, 2)
        return c

    x = inputs(17, B, H, Hk, T, dk, dv, dt)
    a, b = call(wrap(x)), call(on_gpu(x))
    for n in a:
        assert torch.equal(a[n], b[n]), n
    c = on_gpu(x)
    c.update({n: c[n][:1].expand(B, *c[n].shape[1:]) for n in ("q", "k", "v", "g", "beta", "do")})
    full = {n: t.contiguous() if n in ("q", "k", "v", "g", "beta", "do") else t for n, t in c.items()}
    a, b = call(c), call(full)
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_delta_gradients_against_differences():
    # float64 differences of the float64 rule, so that the adjoint itself is tested
    x = {n: t.double() for n, t in inputs(2, 1, 2, 1, 9, 3, 4, F32).items()}
    r = reference(x)

    def loss(y):
        f = reference(y)
        return float((f["o"] * x["do"]).sum() + (f["h_final"] * x["dhT"]).sum())

    for n, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("beta", "dbeta"), ("h0", "dh0")):
        for i in range(0, x[n].numel(), 5):
            step = torch.zeros_like(x[n])
            step.view(-1)[i] = 1e-6
            d = (loss(dict(x, **{n: x[n] + step})) - loss(dict(x, **{n: x[n] - step}))) / 2e-6
            want = float(r[grad].reshape(-1)[i])
            assert abs(d - want) <= 1e-7 * (1 + abs(want)), (n, i, d, want)


def test_delta_is_the_same_every_time_and_in_given_buffers():
    c = on_gpu(inputs(8, 1, 4, 2, 3000, 64, 64, BF16))
    first = call(c)
    for _ in range(3):
        again = call(c)
        for n in first:
            assert torch.equal(first[n], again[n]), n
    a = tuple(c[n] for n in ("q", "k", "v", "g", "beta"))
    dims = (1, 4, 2, 3000, 64, 64, BF16)
    junk = lambda n: torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")  # noqa: E731  (NaN as floats)
    outs = {n: torch.full_like(t, math.nan) for n, t in first.items()}
    o, h_final, saved = gla.gla_delta_fwd(*a, h0=c["h0"], o=outs["o"], h_final=outs["h_final"],
                                          saved=junk(gla.delta_saved_size(*dims)),
                                          workspace=junk(gla.delta_workspace_size(gla.GLA_FWD, *dims)))
    grads = gla.gla_delta_bwd(*a, o, c["do"], saved, dhT=c["dhT"], workspace=junk(gla.delta_workspace_size(gla.GLA_BWD, *dims)),
                              **{n: outs[n] for n in ("dq", "dk", "dv", "dg", "dbeta", "dh0")})
    for n, t in zip(first, (o, h_final) + grads):
        assert t is outs[n] and torch.equal(first[n], t), n


def test_delta_replayed_graphs_and_streams():
    x = [on_gpu(inputs(s, 2, 2, 1, 600, 64, 80, BF16)) for s in (1, 2)]
    want = [call(c) for c in x]
    held = {n: t.clone() for n, t in x[0].items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(held)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = call(held)
    for turn in (1, 0, 1, 0):
        for n in held:
            held[n].copy_(x[turn][n])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n in got:
            assert torch.equal(got[n], want[turn][n]), n
    # two calls at once on two streams
    streams = [torch.cuda.Stream() for _ in range(2)]
    res = []
    for st, c in zip(streams, x):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            res.append([call(c) for _ in range(3)])
    torch.cuda.synchronize()
    for r, w in zip(res, want):
        for one in r:
            for n in w:
                assert torch.equal(one[n], w[n]), n


# ------------------------------------------------------------------------------------ single tokens

@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("B,H,Hk,n,dk,dv", [(1, 1, 1, 1, 1, 1), (2, 4, 2, 1, 128, 128), (3, 2, 1, 3, 100, 50), (5, 3, 3, 2, 16, 17),
                                            (2, 1, 1, 5, 256, 36), (1, 2, 2, 9, 64, 300)])
def test_delta_step(B, H, Hk, n, dk, dv, dt):
    x = inputs(B + dk, B, H, Hk, n, dk, dv, dt)
    slots = torch.randperm(B + 3, generator=torch.Generator().manual_seed(1))[:B]
    pool = torch.randn(B + 3, H, dk, dv, generator=torch.Generator().manual_seed(2))
    x["h0"] = pool[slots]
    r = reference(x)
    c, state = on_gpu(x), pool.cuda()
    o = gla.gla_delta_step(c["q"], c["k"], c["v"], c["g"], c["beta"], state, slots=slots.to(torch.int32).cuda())
    # sums of up to 256 terms, 16 a lane, six exchanges: n additions of half a step of float32 each
    tol = math.sqrt(32 * n) * 2.0 ** -24
    near("o", o, r["o"], tol + (2.0 ** -8 / math.sqrt(3) if dt == BF16 else 0), r["size"]["o"])
    near("state", state[slots.cuda()], r["h_final"], tol, r["size"]["last token"])
    rest = [i for i in range(B + 3) if i not in slots.tolist()]
    assert torch.equal(state[rest].cpu(), pool[rest])


def test_delta_step_slots():
    c = on_gpu(inputs(3, 5, 2, 2, 2, 32, 24, F32))
    pool = torch.randn(4, 2, 32, 24).cuda()
    state = pool.clone()
    slots = torch.tensor([2, -1, 2, 9, 0], dtype=torch.int32).cuda()
    a = tuple(c[n] for n in ("q", "k", "v", "g", "beta"))
    o = gla.gla_delta_step(*a, state, slots=slots)
    one = pool.clone()
    want = gla.gla_delta_step(*(t[[0, 4]] for t in a), one, slots=torch.tensor([2, 0], dtype=torch.int32).cuda())
    assert torch.equal(o[[0, 4]], want) and torch.equal(state, one)
    assert torch.equal(o[1], torch.zeros_like(o[1])) and torch.isnan(o[2]).all() and torch.isnan(o[3]).all()
    assert torch.equal(state[1], pool[1]) and torch.equal(state[3], pool[3])


def test_delta_step_reset_drops_what_is_not_finite():
    c = on_gpu(inputs(4, 2, 1, 1, 1, 16, 16, F32))
    c["g"][:] = -math.inf
    state = torch.full((2, 1, 16, 16), math.nan, device="cuda")
    a = tuple(c[n] for n in ("q", "k", "v", "g", "beta"))
    o = gla.gla_delta_step(*a, state)
    clean = torch.zeros_like(state)
    assert torch.equal(gla.gla_delta_step(*a, clean), o) and torch.equal(state, clean)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_delta_prompt_then_tokens(dt):
    # a prompt by chunks, its state into a pool, then token by token: the same as all of it by chunks
    T, n = 150, 12
    x = inputs(21, 2, 4, 2, T + n, 64, 64, dt)
    c = on_gpu(x)
    cut = lambda lo, hi: tuple(c[m][:, :, lo:hi] for m in ("q", "k", "v", "g", "beta"))  # noqa: E731
    want = reference(x)
    o, state, _ = gla.gla_delta_fwd(*cut(0, T), h0=c["h0"], keep_saved=False)
    rows = [o] + [gla.gla_delta_step(*cut(t, t + 1), state) for t in range(T, T + n)]
    near("o", torch.cat(rows, 2), want["o"], share("o only", dt, dt), want["size"]["o"])
    near("state", state, want["h_final"], share("h_final", dt, F32), want["size"]["h_final"])


# --------------------------------------------------------------------------------------- layer norm

def norm_reference(x, w, b, residual, eps, d_normed=None, d_out=None):
    """Values, and for each the size of the terms that were summed."""
    h = x.double() + (0 if residual is None else residual.double())
    mean = h.mean(-1, keepdim=True)
    r = ((h - mean).square().mean(-1, keepdim=True) + eps).rsqrt()
    n = (h - mean) * r
    # the mean is off by steps of the largest addends, not of itself
    n_size = n.abs() + r * h.abs().mean(-1, keepdim=True) + r * h.abs()
    w = torch.ones(h.shape[-1], dtype=torch.float64) if w is None else w.double()
    y = n * w + (0 if b is None else b.double())
    res = {"out": (h, h.abs()), "normed": (y, n_size * w.abs() + (0 if b is None else b.double().abs()))}
    if d_normed is None:
        return res
    dn = d_normed.double()
    e = dn * w
    dh = r * (e - e.mean(-1, keepdim=True) - n * (e * n).mean(-1, keepdim=True))
    size = r * (e.abs() + e.abs().mean(-1, keepdim=True) + 2 * n_size * (e.abs() * n_size).mean(-1, keepdim=True))
    if d_out is not None:
        dh, size = dh + d_out.double(), size + d_out.double().abs()
    res.update(dx=(dh, size), d_residual=(dh, size), dw=((dn * n).sum((0, 1)), (dn.abs() * n_size).sum((0, 1))),
               db=(dn.sum((0, 1)), dn.abs().sum((0, 1))))
    return res


def norm_check(label, got, ref, rows, D):
    """Element by element: a row's sums are chains of at most 8 D / 4096 + 20 additions, each result 16 roundings besides;
    a column's sums add up rows of a workgroup, then the workgroups'."""
    for n, t in got.items():
        if t is None:
            continue
        want, size = ref[n]
        chain = D / 512 + 40 + (rows / 128 + 600 if n in ("dw", "db") else 0)
        half = torch.finfo(t.dtype).eps / 2
        tol = chain * 2.0 ** -24 * size
        tol = tol + half * (want.abs() + tol)
        t = t.cpu().double()
        assert torch.isfinite(t).all(), (label, n)
        over = float(((t - want).abs() - tol).max())
        assert over <= 0, "%s %s: %.3g more than allowed" % (label, n, over)


NORM_SIZES = [(1, 1, 1), (2, 3, 7), (3, 70, 24), (1, 33, 150), (2, 9, 512), (1, 5, 2048), (1, 70, 2056), (2, 4, 4095),
              (1, 3, 5000), (1, 2, 8192), (1, 3, 12345), (1, 2, 16384), (5, 700, 64)]


@pytest.mark.parametrize("dt,st", [(F32, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("B,T,D", NORM_SIZES)
def test_layernorm(B, T, D, dt, st):
    gen = torch.Generator().manual_seed(D)
    rnd = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    x, dn = (rnd(B, T, D) + 1).to(dt), rnd(B, T, D).to(dt)
    w, b = 1 + 0.1 * rnd(D), 0.1 * rnd(D)
    for res in (True, False):
        residual, d_out = (2 * rnd(B, T, D).to(st), rnd(B, T, D).to(st)) if res else (None, None)
        gpu = lambda t: None if t is None else t.cuda()  # noqa: E731
        f = gla.gla_layernorm_fwd(x.cuda(), w.cuda(), b.cuda(), residual=gpu(residual))
        g = gla.gla_layernorm_bwd(x.cuda(), f, dn.cuda(), w.cuda(), d_out=gpu(d_out), residual=gpu(residual))
        ref = norm_reference(x, w, b, residual, 1e-5, dn, d_out)
        norm_check("res" if res else "plain", {"out": f["out"], "normed": f["normed"], **g}, ref, B * T, D)
        only = gla.gla_layernorm_fwd(x.cuda(), w.cuda(), b.cuda(), residual=gpu(residual), keep_stats=False)
        assert only["mean"] is None and torch.equal(only["normed"], f["normed"])
        assert res == (f["out"] is not None) and (not res or torch.equal(only["out"], f["out"]))
    f = gla.gla_layernorm_fwd(x.cuda())
    g = gla.gla_layernorm_bwd(x.cuda(), f, dn.cuda(), bias=False)
    assert g["dw"] is None and g["db"] is None and g["d_residual"] is None
    norm_check("bare", {"normed": f["normed"], "dx": g["dx"]}, norm_reference(x, None, None, None, 1e-5, dn), B * T, D)


def test_layernorm_views_and_places():
    B, T, D = 3, 40, 100
    gen = torch.Generator().manual_seed(0)
    wide = torch.randn(B, T, 2 * D + 3, generator=gen).cuda()
    x, res = wide[..., 1:1 + D], wide[..., D + 2:2 * D + 2]
    w = torch.rand(D, generator=gen).cuda()
    a = gla.gla_layernorm_fwd(x, w, residual=res)
    b = gla.gla_layernorm_fwd(x.contiguous(), w, residual=res.contiguous())
    assert torch.equal(a["out"], b["out"]) and torch.equal(a["normed"], b["normed"])
    dn, do = x.transpose(0, 1).contiguous().transpose(0, 1), res
    ga = gla.gla_layernorm_bwd(x, a, dn, w, d_out=do, residual=res)
    gb = gla.gla_layernorm_bwd(x.contiguous(), b, dn.contiguous(), w, d_out=do.contiguous(), residual=res.contiguous())
    for n in ga:
        assert torch.equal(ga[n], gb[n]), n
    assert ga["d_residual"] is ga["dx"]
    stream = res.contiguous()
    c = gla.gla_layernorm_fwd(x, w, residual=stream, out=stream, keep_stats=False)
    assert c["out"] is stream and torch.equal(stream, a["out"]) and torch.equal(c["normed"], a["normed"])
    with pytest.raises(ValueError, match="residual's place"):
        gla.gla_layernorm_bwd(x, dict(a, out=stream), dn, w, residual=stream)


def test_layernorm_far_from_zero_and_constant_rows():
    # rows far from zero, whose variance a difference of two sums would lose, and rows without any
    x = 1000 + torch.randn(4, 64, 512, generator=torch.Generator().manual_seed(1))
    norm_check("far", {"normed": gla.gla_layernorm_fwd(x.cuda())["normed"]}, norm_reference(x, None, None, None, 1e-5), 256, 512)
    flat = gla.gla_layernorm_fwd(torch.full((1, 2, 64), 3.0, device="cuda"))
    assert torch.equal(flat["normed"], torch.zeros_like(flat["normed"]))


def test_layernorm_sums_are_the_same_every_time_and_replayed():
    gen = torch.Generator(device="cuda").manual_seed(0)
    x, dn, w = (torch.randn(s, device="cuda", generator=gen) for s in ((2, 9000, 96), (2, 9000, 96), (96,)))
    f = gla.gla_layernorm_fwd(x, w)
    first = gla.gla_layernorm_bwd(x, f, dn, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            again = gla.gla_layernorm_bwd(x, gla.gla_layernorm_fwd(x, w), dn, w)
    for _ in range(3):
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n in ("dx", "dw", "db"):
            assert torch.equal(first[n], again[n]), n


# --------------------------------------------------------------------------------- larger calls, together

def test_offsets_past_32_bits():
    # two sequences whose batch stride passes 2^32 elements, in every input that may be a view
    B, H, T, dk, dv, far = 2, 2, 70, 32, 16, (1 << 32) + 64
    x = on_gpu(inputs(1, B, H, H, T, dk, dv, BF16))
    pool = torch.empty(far + 4 * H * T * 32, dtype=BF16, device="cuda")
    c = dict(x)
    for i, n in enumerate(("q", "k", "v", "do")):
        d = x[n].shape[3]
        c[n] = pool.as_strided((B, H, T, d), (far, T * d, d, 1), i * H * T * 32)
        c[n].copy_(x[n])
    want, got = call(x), call(c)
    for n in want:
        assert torch.equal(want[n], got[n]), n
    rows = pool.as_strided((B, T, 32), (far, 32, 1))
    rows.normal_()
    a, b = gla.gla_layernorm_fwd(rows), gla.gla_layernorm_fwd(rows.contiguous())
    assert torch.equal(a["normed"], b["normed"])


@pytest.mark.parametrize("dt", [F32, BF16])
def test_token_strides_of_a_million(dt):
    # tokens so far apart that a tile's rows are no 32-bit offsets from one base
    T, dk, dv, far = 200, 32, 40, (1 << 20) + 24
    x = on_gpu(inputs(4, 1, 1, 1, T, dk, dv, dt))
    pool, gates = torch.empty(T * far, dtype=dt, device="cuda"), torch.empty(T * far, device="cuda")
    c = dict(x)
    for i, n in enumerate(("q", "k", "v", "do")):
        c[n] = pool.as_strided(x[n].shape, (T * far, T * far, far, 1), i * 64)
        c[n].copy_(x[n])
    for i, n in enumerate(("g", "beta")):
        c[n] = gates.as_strided(x[n].shape, (T * far, T * far, far), i)
        c[n].copy_(x[n])
    want, got = call(x), call(c)
    for n in want:
        assert torch.equal(want[n], got[n]), n


def test_a_block_of_them_together():
    # norm, projections, the rule, and the join with the residual stream: values and the weights' gradients against
    # autograd of the same block in float64
    B, T, H, Hk, d, D = 2, 130, 4, 2, 32, 64
    gen = torch.Generator().manual_seed(5)
    rnd = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    stream, w, b = rnd(B, T, D), 1 + 0.1 * rnd(D), 0.1 * rnd(D)
    proj = {"q": rnd(D, Hk * d) / 8, "k": rnd(D, Hk * d) / 8, "v": rnd(D, H * d) / 8, "wa": rnd(D, H) / 8, "wb": rnd(D, H) / 8}
    back, w_post, d_out = rnd(H * d, D) / 12, 1 + 0.1 * rnd(d), rnd(B, T, D)

    def block(dev, dt, rule, norm, join):
        leaf = {n: t.detach().clone().to(dev, dt).requires_grad_() for n, t in dict(proj, w=w, b=b, back=back, w_post=w_post).items()}
        y = norm(stream.to(dev, dt), leaf["w"], leaf["b"])
        heads = lambda t, n: t.unflatten(-1, (n, -1)).transpose(1, 2)  # noqa: E731
        q, k = (unit(heads(y @ leaf[n], Hk)) for n in "qk")
        g = torch.nn.functional.logsigmoid(y @ leaf["wa"]).transpose(1, 2) / 4
        o = rule(q, k, heads(y @ leaf["v"], H), g, torch.sigmoid(y @ leaf["wb"]).transpose(1, 2))
        out = stream.to(dev, dt) + join(o, leaf["w_post"]) @ leaf["back"]
        out.backward(d_out.to(dev, dt))
        return {"out": out.detach(), **{n: t.grad for n, t in leaf.items()}}

    class Rule(torch.autograd.Function):
        @staticmethod
        def forward(ctx, *a):
            a = tuple(t if t.dim() == 3 else t.contiguous() for t in a)
            o, _, saved = gla.gla_delta_fwd(*a)
            ctx.save_for_backward(*a, o, saved)
            return o

        @staticmethod
        def backward(ctx, do):
            *a, o, saved = ctx.saved_tensors
            return gla.gla_delta_bwd(*a, o, do.contiguous(), saved)[:5]

    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, b):
            f = gla.gla_layernorm_fwd(x, w, b)
            ctx.save_for_backward(x, w)
            ctx.f = f
            return f["normed"]

        @staticmethod
        def backward(ctx, dn):
            x, w = ctx.saved_tensors
            g = gla.gla_layernorm_bwd(x, ctx.f, dn, w)
            return g["dx"], g["dw"], g["db"]

    class Join(torch.autograd.Function):
        @staticmethod
        def forward(ctx, o, w_post):
            ctx.f = gla.gla_join_fwd(o, w_post=w_post)
            ctx.save_for_backward(o, w_post)
            return ctx.f["out"]

        @staticmethod
        def backward(ctx, d):
            o, w_post = ctx.saved_tensors
            g = gla.gla_join_bwd(o, ctx.f, d_out=d, w_post=w_post)
            return g["dy"], g["dw_post"]

    def rule(q, k, v, g, beta):
        q, k = (t.repeat_interleave(H // Hk, 1) for t in (q, k))
        S, o = torch.zeros(B, H, d, d, dtype=torch.float64), []
        for t in range(T):
            A = g[:, :, t, None, None].exp() * S
            e = v[:, :, t] - (k[:, :, t, :, None] * A).sum(2)
            S = A + (beta[:, :, t, None] * k[:, :, t])[..., None] * e[:, :, None]
            o.append((q[:, :, t, :, None] * S).sum(2))
        return torch.stack(o, 2)

    def norm(x, w, b):
        m = x - x.mean(-1, keepdim=True)
        return m / (m.square().mean(-1, keepdim=True) + 1e-5).sqrt() * w + b

    def join(o, w_post):
        n = o / (o.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w_post
        return n.transpose(1, 2).flatten(2)

    want = block("cpu", torch.float64, rule, norm, join)
    got = block("cuda", F32, Rule.apply, Norm.apply, Join.apply)
    for n in want:
        # float32 from end to end: eight operators of at most 192 additions each
        off = float((got[n].cpu().double() - want[n]).norm() / want[n].norm())
        assert off <= 8 * math.sqrt(192 * 12 / 3) * 2.0 ** -24, (n, off)
