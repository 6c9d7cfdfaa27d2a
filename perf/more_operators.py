"""Measured cases of the gated delta rule (chunked forward, training step, single tokens) and of layer norm
joined to the residual stream (forward, training step).

With ``own`` false, ``run`` computes them in elementary torch operations in float32 (log-gates are summed in
float64); with ``own`` true it makes the library's calls.  ``exact`` computes the same outputs in float64 from
the definitions: the delta rule token by token, forward and adjoint.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
DT = {BF16: torch.bfloat16, F32: torch.float32}


def listed():
    return [
        # one token of one sequence through one layer: pure latency
        dict(name="delta_step_b1_h4_128x128", kind="delta_step", B=1, H=4, Hk=4, n=1, dk=128, dv=128, slots=1, dtype=BF16),
        # a full decoding batch, two value heads to a key head, states in a pool addressed by slot
        dict(name="delta_step_b128_h16_128x128", kind="delta_step", B=128, H=16, Hk=8, n=1, dk=128, dv=128, slots=140,
             dtype=BF16),
        # a short prompt
        dict(name="delta_fwd_b1_h4_t50_64x64", kind="delta_fwd", B=1, H=4, Hk=4, T=50, dk=64, dv=64, dtype=BF16,
             ragged=False, docs=0, carry=False, strided=False),
        # prompts of different lengths in a padded batch, q, k and v slices of one fused projection
        dict(name="delta_fwd_b8_h8_t2048_128x128", kind="delta_fwd", B=8, H=8, Hk=8, T=2048, dk=128, dv=128, dtype=BF16,
             ragged=True, docs=0, carry=False, strided=True),
        # one long sequence of few wide heads, continued from a state
        dict(name="delta_fwd_b1_h4_t64k_128x256", kind="delta_fwd", B=1, H=4, Hk=4, T=65536, dk=128, dv=256, dtype=BF16,
             ragged=False, docs=0, carry=True, strided=False),
        # small odd training step in float32
        dict(name="delta_train_b2_h3_t333_48x80", kind="delta_train", B=2, H=3, Hk=3, T=333, dk=48, dv=80, dtype=F32,
             ragged=True, docs=0, carry=True, strided=False),
        # a training step over packed documents, two value heads to a key head
        dict(name="delta_train_b2_h8_t4096_64x128", kind="delta_train", B=2, H=8, Hk=4, T=4096, dk=64, dv=128, dtype=BF16,
             ragged=False, docs=9, carry=False, strided=True),
        # a training step of a 16-head layer over 16k tokens
        dict(name="delta_train_b1_h16_t16k_128x128", kind="delta_train", B=1, H=16, Hk=16, T=16384, dk=128, dv=128,
             dtype=BF16, ragged=False, docs=0, carry=False, strided=False),
        # the residual add and norm of one decoding step
        dict(name="norm_fwd_b32_t1_d2048", kind="norm_fwd", B=32, T=1, D=2048, dtype=BF16, stream=F32, residual=True,
             bias=True),
        # the norm before a block over a 32k-token sequence
        dict(name="norm_fwd_b1_t32k_d2048", kind="norm_fwd", B=1, T=32768, D=2048, dtype=BF16, stream=BF16,
             residual=False, bias=True),
        # odd widths in float32
        dict(name="norm_train_b2_t333_d150", kind="norm_train", B=2, T=333, D=150, dtype=F32, stream=F32, residual=True,
             bias=False),
        # a training step: residual add and norm of 16k tokens
        dict(name="norm_train_b1_t16k_d2048", kind="norm_train", B=1, T=16384, D=2048, dtype=BF16, stream=BF16,
             residual=True, bias=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["delta_step", "delta_fwd", "delta_fwd", "delta_train", "delta_train", "norm_fwd", "norm_train"])
    dtype = rng.choice([BF16, BF16, F32])
    H = rng.choice([1, 2, 3, 4, 6, 8, 16])
    Hk = rng.choice([n for n in range(1, H + 1) if H % n == 0 and n * 4 >= H])
    dk, dv = rng.choice([16, 32, 48, 64, 100, 128, 128]), rng.choice([16, 32, 64, 80, 100, 128, 128, 256])
    if kind == "delta_step":
        B = _log_int(rng, 1, 96)
        return dict(kind=kind, B=B, H=H, Hk=Hk, n=rng.choice([1, 1, 1, 2, 3, 5]), dk=dk, dv=min(dv, 128),
                    slots=B + rng.randrange(0, 16), dtype=dtype)
    if kind in ("delta_fwd", "delta_train"):
        B = _log_int(rng, 1, 8)
        most = (1 << 25 if kind == "delta_train" else 1 << 26) // (2 if dtype == F32 else 1)
        T = _log_int(rng, 1, max(2, min(16384 if kind == "delta_train" else 65536, most // (B * H * max(dk, dv)))))
        return dict(kind=kind, B=B, H=H, Hk=Hk, T=T, dk=dk, dv=dv, dtype=dtype, ragged=rng.random() < 0.4,
                    docs=rng.choice([0, 0, 5]), carry=rng.random() < 0.5, strided=rng.random() < 0.4)
    D = _log_int(rng, 16, 8192)
    if rng.random() < 0.6:
        D = max(8, D // 8 * 8)
    B = _log_int(rng, 1, 32)
    c = dict(kind=kind, B=B, T=_log_int(rng, 1, max(2, (1 << 25) // (B * D))), D=D, dtype=dtype,
             stream=rng.choice([dtype, F32]), residual=rng.random() < 0.6, bias=rng.random() < 0.7)
    if not c["residual"]:
        c["stream"] = dtype
    return c


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
    c, dt = dict(case), DT[case["dtype"]]
    s = {"c": c}
    if c["kind"].startswith("norm"):
        B, T, D, st = c["B"], c["T"], c["D"], DT[c["stream"]]
        s["x"] = (rnd(B, T, D) + 0.3).to(dt)
        s["residual"] = (2 * rnd(B, T, D)).to(st) if c["residual"] else None
        s["w"] = 1 + 0.1 * rnd(D)
        s["b"] = 0.1 * rnd(D) if c["bias"] else None
        if c["kind"] == "norm_train":
            s["d_normed"] = rnd(B, T, D).to(dt)
            s["d_out"] = rnd(B, T, D).to(st) if c["residual"] else None
        return s
    B, H, Hk, dk, dv = c["B"], c["H"], c["Hk"], c["dk"], c["dv"]
    T = c["n"] if c["kind"] == "delta_step" else c["T"]
    unit = lambda t: t * torch.rsqrt(t.square().sum(-1, keepdim=True) + 1e-6)  # noqa: E731
    if c.get("strided"):  # one projection's output [B, T, heads side by side], seen as [B, heads, T, d]
        wide = rnd(B, T, 2 * Hk * dk + H * dv)
        wide[..., :2 * Hk * dk] = unit(wide[..., :2 * Hk * dk].reshape(B, T, 2 * Hk, dk)).reshape(B, T, 2 * Hk * dk)
        wide = wide.to(dt)
        cut = lambda at, n, d: wide[..., at:at + n * d].unflatten(-1, (n, d)).transpose(1, 2)  # noqa: E731
        s["q"], s["k"], s["v"] = cut(0, Hk, dk), cut(Hk * dk, Hk, dk), cut(2 * Hk * dk, H, dv)
    else:
        s["q"], s["k"], s["v"] = unit(rnd(B, Hk, T, dk)).to(dt), unit(rnd(B, Hk, T, dk)).to(dt), rnd(B, H, T, dv).to(dt)
    # decays about 0.95 a token, half of the input written; both as a projection gives them, heads last
    s["g"] = (torch.nn.functional.logsigmoid(rnd(B, T, H)) / 16).transpose(1, 2)
    s["beta"] = torch.sigmoid(rnd(B, T, H)).transpose(1, 2)
    if c["kind"] == "delta_step":
        s["state"] = 0.3 * rnd(c["slots"], H, dk, dv)
        s["slots"] = torch.randperm(c["slots"], device="cuda", generator=gen)[:B].to(torch.int32)
        return s
    if c["docs"]:
        s["g"][:, :, torch.randint(0, T, (c["docs"],), device="cuda", generator=gen)] = -math.inf
    s["h0"] = 0.3 * rnd(B, H, dk, dv) if c["carry"] else None
    s["lens"] = None
    if c["ragged"]:
        s["lens"] = torch.randint(0, T + 1, (B,), device="cuda", generator=gen, dtype=torch.int32)
        s["lens"][0] = T
    if c["kind"] == "delta_train":
        s["do"] = rnd(B, H, T, dv).to(dt)
        s["dhT"] = 0.3 * rnd(B, H, dk, dv) if c["carry"] else None
    return s


EPS = 1e-5


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from sequence_state_scan_amd import gla

    c = s["c"]
    if c["kind"] == "delta_step":
        o = gla.gla_delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], slots=s["slots"])
        return {"o": o, "state": s["state"]}
    if c["kind"] == "delta_fwd":
        o, h_final, _ = gla.gla_delta_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], h0=s["h0"], lens=s["lens"],
                                          keep_saved=False)
        return {"o": o, "h_final": h_final}
    if c["kind"] == "delta_train":
        a = (s["q"], s["k"], s["v"], s["g"], s["beta"])
        o, h_final, saved = gla.gla_delta_fwd(*a, h0=s["h0"], lens=s["lens"])
        dq, dk, dv, dg, dbeta, dh0 = gla.gla_delta_bwd(*a, o, s["do"], saved, lens=s["lens"], dhT=s["dhT"])
        return {"o": o, "h_final": h_final, "dq": dq, "dk": dk, "dv": dv, "dg": dg, "dbeta": dbeta, "dh0": dh0}
    if c["kind"] == "norm_fwd":
        f = gla.gla_layernorm_fwd(s["x"], s["w"], s["b"], residual=s["residual"], eps=EPS, keep_stats=False)
        return {"out": f["out"], "normed": f["normed"]}
    f = gla.gla_layernorm_fwd(s["x"], s["w"], s["b"], residual=s["residual"], eps=EPS)
    b = gla.gla_layernorm_bwd(s["x"], f, s["d_normed"], s["w"], d_out=s["d_out"], residual=s["residual"],
                              bias=s["b"] is not None)
    return {"out": f["out"], "normed": f["normed"], "dx": b["dx"], "d_residual": b["d_residual"], "dw": b["dw"],
            "db": b["db"]}


# ---------------------------------------------------------------------------------- plain forms

CHUNK = 64


def _unit_lower_inverse(L):
    """The inverse of unit lower triangular matrices (a power of 2 wide): diagonal blocks joined two and two."""
    n, size = L.shape[-1], 1
    inv = torch.ones(L.shape[:-1] + (1, 1), device=L.device, dtype=L.dtype)  # [..., blocks, size, size]
    while size < n:
        even = torch.arange(0, n // size, 2, device=L.device)
        blocks = L.unflatten(-2, (n // size, size)).unflatten(-1, (n // size, size)).transpose(-3, -2)
        a, d = inv[..., 0::2, :, :], inv[..., 1::2, :, :]
        below = -(d @ blocks[..., even + 1, even, :, :] @ a)
        inv = torch.cat([torch.cat([a, torch.zeros_like(a)], -1), torch.cat([below, d], -1)], -2)
        size *= 2
    return inv[..., 0, :, :]


def _state_scan(M, U):
    """X_n = M_n X_{n-1} + U_n along dim 2 from zero: pairs combined, the halved sequence scanned, spread back."""
    N = U.shape[2]
    if N == 1:
        return U
    even = slice(0, N - 1, 2)
    odd = _state_scan(M[:, :, 1::2] @ M[:, :, even], M[:, :, 1::2] @ U[:, :, even] + U[:, :, 1::2])
    X = torch.empty_like(U)
    X[:, :, 1::2] = odd
    X[:, :, 0] = U[:, :, 0]
    X[:, :, 2::2] = M[:, :, 2::2] @ odd[:, :, :(N - 1) // 2] + U[:, :, 2::2]
    return X


def _chunks(t, N):
    """[B, H, T, ...] in float32, padded at the end with zeros, as [B, H, N, CHUNK, ...]."""
    T = t.shape[2]
    out = torch.zeros(t.shape[:2] + (N * CHUNK,) + t.shape[3:], device=t.device, dtype=torch.float32)
    out[:, :, :T] = t
    return out.unflatten(2, (N, CHUNK))


def _delta_plain(s, train):
    c, dt = s["c"], s["q"].dtype
    B, H, T, dk, dv = c["B"], c["H"], c["T"], c["dk"], c["dv"]
    G, N = H // c["Hk"], (T + CHUNK - 1) // CHUNK
    q, k = (_chunks(s[n].repeat_interleave(G, 1), N) for n in "qk")
    v, b, g = _chunks(s["v"], N), _chunks(s["beta"], N), _chunks(s["g"].clamp(min=-200.0), N)
    do = _chunks(s["do"], N) if train else None
    live = None
    if s["lens"] is not None:  # behind a sequence's end nothing is read or written
        live = (torch.arange(N * CHUNK, device=q.device) < s["lens"][:, None]).view(B, 1, N, CHUNK)
        q, k, v = (torch.where(live[..., None], t, 0.0) for t in (q, k, v))
        b, g = torch.where(live, b, 0.0), torch.where(live, g, 0.0)
        do = torch.where(live[..., None], do, 0.0) if train else None
    b = b[..., None]
    cg = torch.cumsum(g.double(), -1)
    low = torch.ones(CHUNK, CHUNK, device=q.device, dtype=torch.float32).tril()
    E = torch.exp((cg[..., :, None] - cg[..., None, :]).clamp(max=0)).float() * low  # decay from j to i
    lead, late = torch.exp(cg).float()[..., None], torch.exp(cg[..., -1:] - cg).float()[..., None]
    whole = lead[..., -1:, :]
    kT = k.transpose(-1, -2)
    eye = torch.eye(CHUNK, device=q.device)
    R = _unit_lower_inverse(eye + b * (k @ kT) * E * (1 - eye)) * b.transpose(-1, -2)  # written value = R (v - lead k S)
    P = (q @ kT) * E
    kd = (late * k).transpose(-1, -2)
    M = whole * torch.eye(dk, device=q.device) - kd @ (R @ (lead * k))
    U = kd @ (R @ v)
    h0 = s["h0"] if s["h0"] is not None else torch.zeros(B, H, dk, dv, device=q.device)
    first = U.clone()
    first[:, :, 0] += M[:, :, 0] @ h0
    S1 = _state_scan(M, first)
    S0 = torch.cat([h0[:, :, None], S1[:, :, :-1]], 2)
    y = v - lead * (k @ S0)
    w = R @ y
    o = lead * (q @ S0) + P @ w
    cut = lambda t: t.flatten(2, 3)[:, :, :T]  # noqa: E731
    res = {"o": cut(o).to(dt), "h_final": S1[:, :, -1].clone()}
    if not train:
        return res
    # D: gradient of the state leaving a chunk
    dhT = s["dhT"] if s["dhT"] is not None else torch.zeros(B, H, dk, dv, device=q.device)
    RT = R.transpose(-1, -2)
    PdO = P.transpose(-1, -2) @ do
    V = (lead * q).transpose(-1, -2) @ do - (lead * k).transpose(-1, -2) @ (RT @ PdO)
    MT = M.transpose(-1, -2)
    V[:, :, -1] += MT[:, :, -1] @ dhT
    D0 = _state_scan(MT.flip(2), V.flip(2)).flip(2)
    D = torch.cat([D0[:, :, 1:], dhT[:, :, None]], 2)
    dw = PdO + late * (k @ D)
    dy = RT @ dw                                            # the gradient of v
    kw = (k @ kT) * E * (1 - eye)
    dbeta = ((dw - kw.transpose(-1, -2) @ dy) * (y - kw @ w)).sum(-1)
    dkk = -(dy @ w.transpose(-1, -2)) * E * (1 - eye)
    dP = (do @ w.transpose(-1, -2)) * E
    dq = lead * (do @ S0.transpose(-1, -2)) + dP @ k
    dkey = dP.transpose(-1, -2) @ q + (dkk + dkk.transpose(-1, -2)) @ k - lead * (dy @ S0.transpose(-1, -2)) + \
        late * (w @ D.transpose(-1, -2))
    at = (do * o - dy * v).sum(-1)
    at[..., -1] += (S1 * D).sum((-1, -2))
    dg = torch.flip(torch.cumsum(torch.flip(at, [-1]), -1), [-1])
    dg = torch.where(torch.exp(g) == 0, 0.0, dg)
    if live is not None:
        dg, dbeta = torch.where(live, dg, 0.0), torch.where(live, dbeta, 0.0)
    heads = lambda t: cut(t).unflatten(1, (H // G, G)).sum(2).to(dt)  # noqa: E731
    return dict(res, dq=heads(dq), dk=heads(dkey), dv=cut(dy).to(dt), dg=cut(dg).contiguous(),
                dbeta=cut(dbeta).contiguous(), dh0=D0[:, :, 0].clone())


def _delta_step_plain(s):
    c = s["c"]
    G, at = c["H"] // c["Hk"], s["slots"].long()
    q, k, v = s["q"].float().repeat_interleave(G, 1), s["k"].float().repeat_interleave(G, 1), s["v"].float()
    a, beta, S, o = torch.exp(s["g"]), s["beta"], s["state"][at], []
    for t in range(c["n"]):
        S = a[:, :, t, None, None] * S
        w = beta[:, :, t, None] * (v[:, :, t] - (k[:, :, t, :, None] * S).sum(2))
        S = S + k[:, :, t, :, None] * w[:, :, None, :]
        o.append((q[:, :, t, :, None] * S).sum(2))
    s["state"][at] = S
    return {"o": torch.stack(o, 2).to(s["q"].dtype), "state": s["state"]}


def _norm_plain(s, train):
    dt = s["x"].dtype
    x = s["x"].float()
    h = x if s["residual"] is None else x + s["residual"].float()
    mid = h - h.mean(-1, keepdim=True)
    r = torch.rsqrt(mid.square().mean(-1, keepdim=True) + EPS)
    n = mid * r
    y = n * s["w"]
    if s["b"] is not None:
        y = y + s["b"]
    res = {"out": None if s["residual"] is None else h.to(s["residual"].dtype), "normed": y.to(dt)}
    if not train:
        return res
    dn = s["d_normed"].float()
    e = dn * s["w"]
    dh = r * (e - e.mean(-1, keepdim=True) - n * (e * n).mean(-1, keepdim=True))
    if s["d_out"] is not None:
        dh = dh + s["d_out"].float()
    return dict(res, dx=dh.to(dt), d_residual=None if s["residual"] is None else dh.to(s["residual"].dtype),
                dw=(dn * n).sum((0, 1)), db=dn.sum((0, 1)) if s["b"] is not None else None)


def _run_plain(s):
    kind = s["c"]["kind"]
    if kind == "delta_step":
        return _delta_step_plain(s)
    if kind in ("delta_fwd", "delta_train"):
        return _delta_plain(s, kind == "delta_train")
    return _norm_plain(s, kind == "norm_train")


# ------------------------------------------------------------------------------------ the measure

def work(case):
    c = case
    e = 2 if c["dtype"] == BF16 else 4
    if c["kind"].startswith("norm"):
        n, st = c["B"] * c["T"] * c["D"], (2 if c["stream"] == BF16 else 4) if c["residual"] else 0
        if c["kind"] == "norm_fwd":
            return {"bytes": n * (2 * e + 2 * st), "flops": 9 * n}
        return {"bytes": n * (2 * e + 2 * st + 2 * e + 2 * st), "flops": 25 * n}
    T = c["n"] if c["kind"] == "delta_step" else c["T"]
    B, H, dk, dv = c["B"], c["H"], c["dk"], c["dv"]
    qk, v, gate, state = B * c["Hk"] * T * dk * e, B * H * T * dv * e, B * H * T * 4, B * H * dk * dv * 4
    fwd = {"bytes": 2 * qk + 2 * v + 2 * gate + state, "flops": 7 * B * H * T * dk * dv}
    if c["kind"] == "delta_step" or (c["kind"] == "delta_fwd" and c["carry"]):
        return {"bytes": fwd["bytes"] + state, "flops": fwd["flops"]}
    if c["kind"] == "delta_fwd":
        return fwd
    edge = state * (4 if c["carry"] else 2)
    return {"bytes": 4 * qk + 4 * v + 4 * gate + edge, "flops": 3 * fwd["flops"]}


# -------------------------------------------------------------------------------------- in 64 bits

def _token(S, k, v, a, beta):
    """The decayed state, the error of its prediction of v, and the state after the token."""
    A = a[..., None, None] * S
    err = v - torch.matmul(k[..., None, :], A)[..., 0, :]
    return A, err, A + (beta[..., None] * k)[..., :, None] * err[..., None, :]


def _delta_definition(s, train):
    c = s["c"]
    B, H, T, dk, dv = c["B"], c["H"], c["T"], c["dk"], c["dv"]
    G = H // c["Hk"]
    tok = lambda t: t.double().permute(2, 0, 1, *range(3, t.dim())).contiguous()  # noqa: E731  (tokens first)
    q, k = (tok(s[n].repeat_interleave(G, 1)) for n in "qk")
    v, a, beta = tok(s["v"]), tok(s["g"]).exp(), tok(s["beta"])
    if s["lens"] is not None:
        past = (torch.arange(T, device=v.device)[:, None] >= s["lens"][None, :]).view(T, B, 1).expand(T, B, H)
        a, beta, q = a.masked_fill(past, 1.0), beta.masked_fill(past, 0.0), q.masked_fill(past[..., None], 0.0)
    zero = torch.zeros(B, H, dk, dv, device=v.device, dtype=torch.float64)
    S = zero if s["h0"] is None else s["h0"].double()
    o, marks, every = torch.empty_like(v), [], 128
    for t in range(T):
        if t % every == 0:
            marks.append(S)
        S = _token(S, k[t], v[t], a[t], beta[t])[2]
        o[t] = torch.matmul(q[t][..., None, :], S)[..., 0, :]
    back = lambda t: t.permute(1, 2, 0, *range(3, t.dim()))  # noqa: E731
    res = {"o": back(o), "h_final": S}
    if not train:
        return res
    do = tok(s["do"])
    if s["lens"] is not None:
        do = do.masked_fill(past[..., None], 0.0)
    D = zero if s["dhT"] is None else s["dhT"].double()
    dq, dkey, dval, da, db = (torch.empty_like(t) for t in (q, k, v, a, beta))
    for m in range(len(marks) - 1, -1, -1):
        S, kept = marks[m], []
        for t in range(m * every, min(T, (m + 1) * every)):
            A, err, after = _token(S, k[t], v[t], a[t], beta[t])
            kept.append((S, A, err, after))
            S = after
        for t in range(min(T, (m + 1) * every) - 1, m * every - 1, -1):
            S, A, err, after = kept.pop()
            dq[t] = torch.matmul(after, do[t][..., None])[..., 0]
            D = D + q[t][..., :, None] * do[t][..., None, :]
            De = torch.matmul(D, err[..., None])[..., 0]
            Dk = torch.matmul(k[t][..., None, :], D)[..., 0, :]
            db[t] = (k[t] * De).sum(-1)
            derr = beta[t][..., None] * Dk
            dval[t] = derr
            dkey[t] = beta[t][..., None] * De - torch.matmul(A, derr[..., None])[..., 0]
            D = D - k[t][..., :, None] * derr[..., None, :]
            da[t] = (D * S).sum((-1, -2))
            D = a[t][..., None, None] * D
    dg = da * a
    if s["lens"] is not None:
        dg, db = dg.masked_fill(past, 0.0), db.masked_fill(past, 0.0)
        dkey = dkey.masked_fill(past[..., None], 0.0)
    heads = lambda t: back(t).unflatten(1, (H // G, G)).sum(2)  # noqa: E731
    return dict(res, dq=heads(dq), dk=heads(dkey), dv=back(dval), dg=back(dg), dbeta=back(db), dh0=D)


def exact(case, seed):
    kind = case["kind"]
    if kind == "delta_train" and case["T"] > 20000:  # the adjoint token by token would take too long
        return None
    s = prepare(case, seed)
    if kind in ("delta_fwd", "delta_train"):
        return _delta_definition(s, kind == "delta_train")
    if kind == "delta_step":
        at, G = s["slots"].long(), case["H"] // case["Hk"]
        q, k = (s[n].double().repeat_interleave(G, 1) for n in "qk")
        state, o = s["state"].double(), []
        S = state[at]
        for t in range(case["n"]):
            S = _token(S, k[:, :, t], s["v"][:, :, t].double(), s["g"][:, :, t].double().exp(),
                       s["beta"][:, :, t].double())[2]
            o.append(torch.matmul(q[:, :, t, None, :], S)[..., 0, :])
        state[at] = S
        return {"o": torch.stack(o, 2), "state": state}
    train = kind == "norm_train"
    leaf = {n: None if s[n] is None else s[n].double().requires_grad_(train) for n in ("x", "residual", "w", "b")}
    h = leaf["x"] if leaf["residual"] is None else leaf["x"] + leaf["residual"]
    mean = h.sum(-1, keepdim=True) / h.shape[-1]
    y = (h - mean) / ((h - mean).pow(2).sum(-1, keepdim=True) / h.shape[-1] + EPS).sqrt() * leaf["w"]
    if leaf["b"] is not None:
        y = y + leaf["b"]
    res = {"out": None if leaf["residual"] is None else h.detach(), "normed": y.detach()}
    if not train:
        return res
    total = (y * s["d_normed"].double()).sum()
    if s["d_out"] is not None:
        total = total + (h * s["d_out"].double()).sum()
    have = [n for n in leaf if leaf[n] is not None]
    grads = dict(zip(have, torch.autograd.grad(total, [leaf[n] for n in have])))
    return dict(res, dx=grads["x"], d_residual=grads.get("residual"), dw=grads["w"], db=grads.get("b"))
