"""Measured cases of the recurrent-block operators: the elementwise gated linear recurrence (forward,
training step, single token), the join of a block's output with the residual stream (head norm, gate,
residual scale and add, the next block's norm), and gated linear attention's single-token step.

With ``own`` false, ``run`` computes them in elementary torch operations in float32; with ``own``
true it makes the library's calls.  ``exact`` computes the same outputs in float64, from the
definitions (gradients by differentiating them).
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
DT = {BF16: torch.bfloat16, F32: torch.float32}


def listed():
    return [
        # one token of one sequence through one recurrent layer: pure latency
        dict(name="recur_step_b1_d2048", kind="recur_step", B=1, D=2048, slots=1, mode="lerp", dtype=BF16),
        # a full decoding batch, states in a pool addressed by slot
        dict(name="recur_step_b256_d4096", kind="recur_step", B=256, D=4096, slots=320, mode="norm", dtype=BF16),
        # prompts of different lengths in a padded batch, x a slice of a fused projection
        dict(name="recur_fwd_b8_t2048_d2560", kind="recur_fwd", B=8, T=2048, D=2560, mode="norm", dtype=BF16,
             ragged=True, docs=0, carry=False, strided=True),
        # one very long sequence of packed documents (each starts with a reset)
        dict(name="recur_fwd_b1_t256k_d1024", kind="recur_fwd", B=1, T=262144, D=1024, mode="lerp", dtype=BF16,
             ragged=False, docs=37, carry=True, strided=False),
        # small odd training step in float32
        dict(name="recur_train_b2_t777_d100", kind="recur_train", B=2, T=777, D=100, mode="plain", dtype=F32,
             ragged=True, docs=0, carry=True, strided=False),
        # a training step at ordinary sizes
        dict(name="recur_train_b4_t4096_d2048", kind="recur_train", B=4, T=4096, D=2048, mode="norm", dtype=BF16,
             ragged=False, docs=9, carry=False, strided=True),
        # gated linear attention's output norm and gate over a 32k-token sequence, 4 heads of 256
        dict(name="join_fwd_h4_t32k_d256", kind="join_fwd", B=1, H=4, T=32768, d=256, dtype=BF16, stream=BF16,
             post=True, gate="silu", residual=False, scale=False, pre=False),
        # the residual add and next norm of one decoding step
        dict(name="join_fwd_b32_t1_d2048", kind="join_fwd", B=32, H=1, T=1, d=2048, dtype=BF16, stream=F32,
             post=True, gate="", residual=True, scale=True, pre=True),
        # odd widths, everything on, float32
        dict(name="join_train_b2_h3_t333_d50", kind="join_train", B=2, H=3, T=333, d=50, dtype=F32, stream=F32,
             post=True, gate="sigmoid", residual=True, scale=True, pre=True),
        # a training step of a 16-head block over 16k tokens, everything on
        dict(name="join_train_h16_t16k_d128", kind="join_train", B=1, H=16, T=16384, d=128, dtype=BF16, stream=BF16,
             post=True, gate="silu", residual=True, scale=True, pre=True),
        # one token of one sequence, 4 heads of 128 x 256
        dict(name="step_b1_h4_128x256", kind="step", B=1, H=4, n=1, dk=128, dv=256, slots=1, dtype=BF16),
        # a full decoding batch of 16 heads of 128 x 128
        dict(name="step_b128_h16_128x128", kind="step", B=128, H=16, n=1, dk=128, dv=128, slots=140, dtype=BF16),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["recur_step", "recur_fwd", "recur_fwd", "recur_train", "recur_train", "join_fwd", "join_train",
                       "join_train", "step", "step"])
    dtype = rng.choice([BF16, BF16, F32])
    mode = rng.choice(["plain", "lerp", "norm"])
    if kind == "recur_step":
        B = _log_int(rng, 1, 256)
        return dict(kind=kind, B=B, D=_log_int(rng, 16, 4096), slots=B + rng.randrange(0, 64), mode=mode, dtype=dtype)
    if kind in ("recur_fwd", "recur_train"):
        most = 1 << (27 if kind == "recur_fwd" else 25)
        B, D = _log_int(rng, 1, 16), _log_int(rng, 16, 4096)
        if rng.random() < 0.6:
            D = max(8, D // 8 * 8)
        T = _log_int(rng, 1, max(2, min(262144, most // (B * D))))
        return dict(kind=kind, B=B, T=T, D=D, mode=mode, dtype=dtype, ragged=rng.random() < 0.4,
                    docs=rng.choice([0, 0, 5]), carry=rng.random() < 0.5, strided=rng.random() < 0.4)
    if kind in ("join_fwd", "join_train"):
        H = rng.choice([1, 1, 2, 3, 4, 8, 16])
        d = _log_int(rng, 16, 256) if H > 1 else _log_int(rng, 16, 8192)
        if rng.random() < 0.7:
            d = max(8, d // 8 * 8)
        B = _log_int(rng, 1, 32)
        T = _log_int(rng, 1, max(2, (1 << 24) // (B * H * d)))
        c = dict(kind=kind, B=B, H=H, T=T, d=d, dtype=dtype, stream=rng.choice([dtype, F32]), post=rng.random() < 0.8,
                 gate=rng.choice(["", "silu", "sigmoid"]), residual=rng.random() < 0.7, scale=rng.random() < 0.5,
                 pre=rng.random() < 0.7)
        if not c["residual"]:
            c["stream"] = dtype
        return c
    B, H = _log_int(rng, 1, 96), rng.choice([1, 2, 3, 4, 8, 16])
    return dict(kind=kind, B=B, H=H, n=rng.choice([1, 1, 1, 2, 3, 5, 8]), dk=rng.choice([16, 32, 64, 100, 128]),
                dv=rng.choice([16, 32, 64, 96, 128]), slots=B + rng.randrange(0, 16), dtype=dtype)


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
    gates = lambda *s: torch.nn.functional.logsigmoid(rnd(*s)) / 16  # noqa: E731  (decays about 0.95 a token)
    c, dt = dict(case), DT[case["dtype"]]
    s = {"c": c}
    kind = c["kind"]
    if kind == "recur_step":
        B, D = c["B"], c["D"]
        s["x"], s["g"], s["state"] = rnd(B, D).to(dt), gates(B, D), rnd(c["slots"], D)
        s["slots"] = torch.randperm(c["slots"], device="cuda", generator=gen)[:B].to(torch.int32)
    elif kind in ("recur_fwd", "recur_train"):
        B, T, D = c["B"], c["T"], c["D"]
        s["x"] = rnd(B, T, 2 * D).to(dt)[..., :D] if c["strided"] else rnd(B, T, D).to(dt)
        s["g"] = gates(B, T, D)
        if c["docs"]:
            s["g"][:, torch.randint(0, T, (c["docs"],), device="cuda", generator=gen)] = -math.inf
        s["h0"] = rnd(B, D) if c["carry"] else None
        s["lens"] = None
        if c["ragged"]:
            s["lens"] = torch.randint(0, T + 1, (B,), device="cuda", generator=gen, dtype=torch.int32)
            s["lens"][0] = T
        if kind == "recur_train":
            s["dh"] = rnd(B, T, D).to(dt)
            s["dhT"] = rnd(B, D) if c["carry"] else None
    elif kind in ("join_fwd", "join_train"):
        B, H, T, d = c["B"], c["H"], c["T"], c["d"]
        D, st = H * d, DT[c["stream"]]
        s["y"] = rnd(B, H, T, d).to(dt)
        s["z"] = rnd(B, T, D).to(dt) if c["gate"] else None
        s["w_post"] = 1 + 0.1 * rnd(d) if c["post"] else None
        s["residual"] = (2 * rnd(B, T, D)).to(st) if c["residual"] else None
        s["scale"] = 0.5 + 0.1 * rnd(D) if c["scale"] else None
        s["w_pre"] = 1 + 0.1 * rnd(D) if c["pre"] else None
        if kind == "join_train":
            s["d_out"] = rnd(B, T, D).to(st)
            s["d_normed"] = rnd(B, T, D).to(dt) if c["pre"] else None
    else:
        B, H, n, dk, dv = c["B"], c["H"], c["n"], c["dk"], c["dv"]
        r = 1 / math.sqrt(dk)
        s["q"], s["k"], s["v"] = (rnd(B, H, n, dk) * r).to(dt), (rnd(B, H, n, dk) * r).to(dt), rnd(B, H, n, dv).to(dt)
        s["g"], s["state"] = gates(B, H, n, dk), rnd(c["slots"], H, dk, dv) * r
        s["slots"] = torch.randperm(c["slots"], device="cuda", generator=gen)[:B].to(torch.int32)
    return s


EPS = 1e-6


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from sequence_state_scan_amd import gla

    c = s["c"]
    kind = c["kind"]
    if kind == "recur_step":
        return {"h": gla.gla_recur_step(s["x"], s["g"], s["state"], slots=s["slots"], mode=c["mode"]), "state": s["state"]}
    if kind == "recur_fwd":
        h, _, h_final = gla.gla_recur_fwd(s["x"], s["g"], h0=s["h0"], lens=s["lens"], mode=c["mode"],
                                          keep_chunk_states=False)
        return {"h": h, "h_final": h_final}
    if kind == "recur_train":
        h, chunk_in, h_final = gla.gla_recur_fwd(s["x"], s["g"], h0=s["h0"], lens=s["lens"], mode=c["mode"])
        dx, dg, dh0 = gla.gla_recur_bwd(s["x"], s["g"], s["dh"], chunk_in, lens=s["lens"], dhT=s["dhT"], mode=c["mode"])
        return {"h": h, "h_final": h_final, "dx": dx, "dg": dg, "dh0": dh0}
    if kind == "join_fwd":
        f = gla.gla_join_fwd(s["y"], z=s["z"], w_post=s["w_post"], residual=s["residual"], scale=s["scale"],
                             w_pre=s["w_pre"], act=c["gate"] or "silu", eps=EPS, keep_rstd=False)
        return {"out": f["out"], "normed": f["normed"]}
    if kind == "join_train":
        f = gla.gla_join_fwd(s["y"], z=s["z"], w_post=s["w_post"], residual=s["residual"], scale=s["scale"],
                             w_pre=s["w_pre"], act=c["gate"] or "silu", eps=EPS)
        b = gla.gla_join_bwd(s["y"], f, d_out=s["d_out"], d_normed=s["d_normed"], z=s["z"], w_post=s["w_post"],
                             residual=s["residual"], scale=s["scale"], w_pre=s["w_pre"], act=c["gate"] or "silu")
        return {"out": f["out"], "normed": f["normed"], "dy": b["dy"], "dz": b["dz"], "d_residual": b["d_residual"],
                "dw_post": b["dw_post"], "dscale": b["dscale"], "dw_pre": b["dw_pre"]}
    o = gla.gla_step(s["q"], s["k"], s["v"], s["g"], s["state"], slots=s["slots"])
    return {"o": o, "state": s["state"]}


# ---------------------------------------------------------------------------------- plain forms

def _beta(g, mode):
    """The input's factor and its derivative by g."""
    if mode == "plain":
        return torch.ones_like(g), torch.zeros_like(g)
    if mode == "lerp":
        return -torch.expm1(g), -torch.exp(g)
    b = torch.sqrt(-torch.expm1(2 * g))
    return b, torch.where(b > 0, -torch.exp(2 * g) / b, 0.0)


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 from zero: pairs combined, the halved sequence scanned, spread back."""
    T = b.shape[1]
    if T == 1:
        return b
    odd = _scan(a[:, 1::2] * a[:, 0:T - 1:2], a[:, 1::2] * b[:, 0:T - 1:2] + b[:, 1::2])
    h = torch.empty_like(b)
    h[:, 1::2] = odd
    h[:, 0] = b[:, 0]
    h[:, 2::2] = a[:, 2::2] * odd[:, :(T - 1) // 2] + b[:, 2::2]
    return h


def _live(lens, T):
    return None if lens is None else (torch.arange(T, device=lens.device)[None, :] < lens[:, None].long())[..., None]


def _recur_plain(s, train):
    c, x, g = s["c"], s["x"].float(), s["g"]
    B, T, D = x.shape
    live = _live(s["lens"], T)
    a = torch.exp(g)
    beta, dbeta = _beta(g, c["mode"])
    b = beta * x
    if live is not None:  # behind a sequence's end the state stays
        a, b = torch.where(live, a, 1.0), torch.where(live, b, 0.0)
    h0 = s["h0"] if s["h0"] is not None else torch.zeros_like(x[:, 0])
    lead = b.clone()
    lead[:, 0] += a[:, 0] * h0
    h = _scan(a, lead)
    out = {"h": (h if live is None else torch.where(live, h, 0.0)).to(s["x"].dtype), "h_final": h[:, -1].clone()}
    if not train:
        return out
    dh = s["dh"].float()
    if live is not None:
        dh = torch.where(live, dh, 0.0)
    if s["dhT"] is not None:
        dh = torch.cat([dh[:, :-1], dh[:, -1:] + s["dhT"][:, None]], 1)
    after = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    G = _scan(after.flip(1), dh.flip(1)).flip(1)
    before = torch.cat([h0[:, None], h[:, :-1]], 1)
    dx, dg = beta * G, a * before * G + dbeta * x * G
    if live is not None:
        dx, dg = torch.where(live, dx, 0.0), torch.where(live, dg, 0.0)
    return dict(out, dx=dx.to(s["x"].dtype), dg=dg, dh0=a[:, 0] * G[:, 0])


def _join_plain(s, train):
    c, dt = s["c"], s["y"].dtype
    st = DT[c["stream"]]
    y = s["y"].float()
    B, H, T, d = y.shape
    rows = lambda t: t.transpose(1, 2).reshape(B, T, H * d)  # noqa: E731
    heads = lambda t: t.reshape(B, T, H, d).transpose(1, 2)  # noqa: E731
    ry = torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) if c["post"] else None
    yn = y * ry if c["post"] else y
    u = rows(yn * s["w_post"] if c["post"] else yn)
    z = s["z"].float() if c["gate"] else None
    sig = torch.sigmoid(z) if c["gate"] else None
    act = 1.0 if z is None else z * sig if c["gate"] == "silu" else sig
    m = u * act
    out = m * s["scale"] if c["scale"] else m
    if c["residual"]:
        out = out + s["residual"].float()
    rp = torch.rsqrt(out.square().mean(-1, keepdim=True) + EPS) if c["pre"] else None
    nh = out * rp if c["pre"] else None
    res = {"out": out.to(st), "normed": (nh * s["w_pre"]).to(dt) if c["pre"] else None}
    if not train:
        return res
    do = s["d_out"].float()
    if c["pre"]:
        dn = s["d_normed"].float()
        e = dn * s["w_pre"]
        do = do + rp * (e - nh * (e * nh).mean(-1, keepdim=True))
        res["dw_pre"] = (dn * nh).sum((0, 1))
    else:
        res["dw_pre"] = None
    res["d_residual"] = do.to(st) if c["residual"] else None
    res["dscale"] = (do * m).sum((0, 1)) if c["scale"] else None
    dm = do * s["scale"] if c["scale"] else do
    if c["gate"]:
        slope = sig * (1 + z * (1 - sig)) if c["gate"] == "silu" else sig * (1 - sig)
        res["dz"] = (dm * u * slope).to(dt)
    else:
        res["dz"] = None
    du = heads(dm * act)
    if c["post"]:
        res["dw_post"] = (du * yn).sum((0, 1, 2))
        e = du * s["w_post"]
        dy = ry * (e - yn * (e * yn).mean(-1, keepdim=True))
    else:
        res["dw_post"], dy = None, du
    res["dy"] = dy.to(dt).contiguous()
    return res


def _step_plain(s):
    q, k, v, g = s["q"].float(), s["k"].float(), s["v"].float(), s["g"]
    n = q.shape[2]
    at = s["slots"].long()
    S = s["state"][at]
    if n == 1:
        S = torch.exp(g[:, :, 0, :, None]) * S + k[:, :, 0, :, None] * v[:, :, 0, None, :]
        o = (q[:, :, 0, :, None] * S).sum(2, keepdim=True)
    else:
        cg = torch.cumsum(g, 2)
        w = torch.exp((cg[:, :, :, None] - cg[:, :, None]).clamp(max=0))  # [B, H, t, s, dk]
        w = w * torch.ones(n, n, device=q.device).tril()[:, :, None]
        p = (q[:, :, :, None] * w * k[:, :, None]).sum(-1)
        o = (p[..., None] * v[:, :, None]).sum(3) + ((q * torch.exp(cg))[..., None] * S[:, :, None]).sum(3)
        late = torch.exp(cg[:, :, -1:] - cg) * k
        S = torch.exp(cg[:, :, -1])[..., None] * S + (late[..., None] * v[:, :, :, None]).sum(2)
    s["state"][at] = S
    return {"o": o.to(s["q"].dtype), "state": s["state"]}


def _recur_step_plain(s):
    x, g, at = s["x"].float(), s["g"], s["slots"].long()
    h = torch.exp(g) * s["state"][at] + _beta(g, s["c"]["mode"])[0] * x
    s["state"][at] = h
    return {"h": h.to(s["x"].dtype), "state": s["state"]}


def _run_plain(s):
    kind = s["c"]["kind"]
    if kind == "recur_step":
        return _recur_step_plain(s)
    if kind in ("recur_fwd", "recur_train"):
        return _recur_plain(s, kind == "recur_train")
    if kind in ("join_fwd", "join_train"):
        return _join_plain(s, kind == "join_train")
    return _step_plain(s)


# ------------------------------------------------------------------------------------ the measure

def work(case):
    c = case
    e = 2 if c["dtype"] == BF16 else 4
    kind = c["kind"]
    if kind == "recur_step":
        n = c["B"] * c["D"]
        return {"bytes": n * (2 * e + 12) + 4 * c["B"], "flops": 6 * n}
    if kind in ("recur_fwd", "recur_train"):
        n, edge = c["B"] * c["T"] * c["D"], 4 * c["B"] * c["D"]
        fwd = n * (2 * e + 4) + edge * (1 + c["carry"])
        if kind == "recur_fwd":
            return {"bytes": fwd, "flops": 6 * n}
        return {"bytes": fwd + n * (2 * e + 4) + edge * (1 + c["carry"]), "flops": 18 * n}
    if kind in ("join_fwd", "join_train"):
        n, st = c["B"] * c["T"] * c["H"] * c["d"], 2 if c["stream"] == BF16 else 4
        e_, st_ = e, st
        fwd = e_ + st_ + (e_ if c["gate"] else 0) + (st_ if c["residual"] else 0) + (e_ if c["pre"] else 0)
        if kind == "join_fwd":
            return {"bytes": n * fwd, "flops": 16 * n}
        bwd = e_ + st_ + (e_ if c["gate"] else 0) + (st_ if c["residual"] else 0) + (e_ if c["pre"] else 0)
        return {"bytes": n * (fwd + bwd), "flops": 50 * n}
    h = c["B"] * c["H"]
    return {"bytes": h * (8 * c["dk"] * c["dv"] + c["n"] * (2 * e * c["dk"] + 2 * e * c["dv"] + 4 * c["dk"])),
            "flops": h * c["n"] * 5 * c["dk"] * c["dv"]}


# -------------------------------------------------------------------------------------- in 64 bits

def _doubling(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1: every step doubles the stretch that each position covers."""
    k, T = 1, b.shape[1]
    while k < T:
        b = torch.cat([b[:, :k], a[:, k:] * b[:, :-k] + b[:, k:]], 1)
        a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], 1)
        k *= 2
    return b


def _recur_definition(x, g, h0, lens, mode):
    T = x.shape[1]
    a = g.exp()
    if mode == "plain":
        b = x
    elif mode == "lerp":
        b = -g.expm1() * x
    else:
        b = (-(2 * g).expm1()).sqrt() * x
    if lens is not None:
        past = (torch.arange(T, device=x.device)[None, :] >= lens[:, None].long())[..., None]
        a, b = a.masked_fill(past, 1.0), b.masked_fill(past, 0.0)
    if h0 is not None:
        b = torch.cat([(a[:, :1] * h0[:, None] + b[:, :1]), b[:, 1:]], 1)
    h = _doubling(a, b)
    return (h if lens is None else h.masked_fill(past, 0.0)), h[:, -1]


def _join_definition(c, y, z, w_post, residual, scale, w_pre):
    B, H, T, d = y.shape
    norm = lambda t: t / (t.pow(2).mean(-1, keepdim=True) + EPS).sqrt()  # noqa: E731
    u = norm(y) * w_post if w_post is not None else y
    u = u.permute(0, 2, 1, 3).reshape(B, T, H * d)
    if z is not None:
        u = u / (1 + (-z).exp()) * (z if c["gate"] == "silu" else 1.0)
    if scale is not None:
        u = u * scale
    if residual is not None:
        u = u + residual
    return u, (norm(u) * w_pre if w_pre is not None else None)


def exact(case, seed):
    s = prepare(case, seed)
    c, kind = s["c"], s["c"]["kind"]
    f64 = lambda t: None if t is None else t.double()  # noqa: E731
    if kind == "recur_step":
        at, g = s["slots"].long(), f64(s["g"])
        h, _ = _recur_definition(f64(s["x"])[:, None], g[:, None], f64(s["state"])[at], None, c["mode"])
        state = f64(s["state"])
        state[at] = h[:, 0]
        return {"h": h[:, 0], "state": state}
    if kind == "recur_fwd":
        h, last = _recur_definition(f64(s["x"]), f64(s["g"]), f64(s["h0"]), s["lens"], c["mode"])
        return {"h": h, "h_final": last}
    if kind == "recur_train":
        leaf = {n: f64(s[n]).requires_grad_() for n in ("x", "g")}
        B, T, D = leaf["x"].shape
        h0 = (f64(s["h0"]) if s["h0"] is not None else torch.zeros_like(leaf["x"][:, 0])).detach().requires_grad_()
        h, last = _recur_definition(leaf["x"], leaf["g"], h0, s["lens"], c["mode"])
        total = (h * f64(s["dh"])).sum() + ((last * f64(s["dhT"])).sum() if s["dhT"] is not None else 0)
        dx, dg, dh0 = torch.autograd.grad(total, [leaf["x"], leaf["g"], h0])
        return {"h": h.detach(), "h_final": last.detach(), "dx": dx, "dg": dg, "dh0": dh0}
    if kind in ("join_fwd", "join_train"):
        names = ("y", "z", "w_post", "residual", "scale", "w_pre")
        leaf = {n: None if s[n] is None else f64(s[n]).requires_grad_(kind == "join_train") for n in names}
        out, normed = _join_definition(c, *(leaf[n] for n in names))
        res = {"out": out.detach(), "normed": None if normed is None else normed.detach()}
        if kind == "join_fwd":
            return res
        total = (out * f64(s["d_out"])).sum() + (0 if normed is None else (normed * f64(s["d_normed"])).sum())
        have = [n for n in names if leaf[n] is not None]
        grads = dict(zip(have, torch.autograd.grad(total, [leaf[n] for n in have])))
        for n, to in (("y", "dy"), ("z", "dz"), ("w_post", "dw_post"), ("residual", "d_residual"), ("scale", "dscale"),
                      ("w_pre", "dw_pre")):
            res[to] = grads.get(n)
        return res
    at, state = s["slots"].long(), f64(s["state"])
    q, k, v, a = f64(s["q"]), f64(s["k"]), f64(s["v"]), f64(s["g"]).exp()
    S, o = state[at], []
    for t in range(c["n"]):
        S = a[:, :, t, :, None] * S + torch.einsum("bhi,bhj->bhij", k[:, :, t], v[:, :, t])
        o.append((q[:, :, t, :, None] * S).sum(2))
    state[at] = S
    return {"o": torch.stack(o, 2), "state": state}
