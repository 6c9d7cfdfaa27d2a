"""The size of what dg of the gated delta rule is summed from, for bounds on its error.

A token's dg is the sum, from the token to the next mark (every 256th token, or the end), of o . do - v . dv, and <S, D> at
the mark; the sum from the mark before has to be <S, D> there, and what it is off by goes back to the span's tokens by the
sizes of their terms.  Errors of single products are independent, so a token's terms are the root of the sum of the squares
of o do and v dv, and a mark's of those of S D, each factor by its own terms where it is a sum that cancels; and what comes
back is a share of the whole span's.
"""
import torch

from test_gpu_delta import reference

SPAN = 256
TOKENS = ("q", "k", "v", "g", "beta", "do")


def marks(x):
    """Of every mark, from the start on: <S, D> by products [B, H, dk, dv], and the root of its terms' squares [B, H]."""
    T, out, h0 = x["q"].shape[2], [], x["h0"]
    for at in list(range(0, T, SPAN)) + [T]:
        cut = lambda lo, hi, **kw: {**{n: x[n][:, :, lo:hi] for n in TOKENS}, **kw}  # noqa: E731
        S = s_size = h0.double()
        if at:
            r = reference(cut(0, at, h0=h0, dhT=None))
            S, s_size = r["h_final"], torch.hypot(r["h_final"], r["size"]["h_final"])
        D = d_size = x["dhT"].double()
        if at < T:
            r = reference(cut(at, T, h0=S, dhT=x["dhT"]))
            D, d_size = r["dh0"], torch.hypot(r["dh0"], r["size"]["dh0"])
        out.append((S * D, (s_size.square() * D.square() + S.square() * d_size.square()).sum((-1, -2)).sqrt()))
    return out


def gate_terms(x, r):
    """The root of the squares of dg's terms, [B, H, T]."""
    do, v, T = x["do"].double(), x["v"].double(), x["q"].shape[2]
    o, dv = torch.hypot(r["o"], r["size"]["o"]), torch.hypot(r["dv"], r["size"]["dv"])
    own = ((o * do).square() + (dv * v).square()).sum(-1)
    size = ((r["o"] * do).abs() + (r["dv"] * v).abs()).sum(-1)
    ends, out = [m[1].square() for m in marks(x)], torch.zeros_like(own)
    back = lambda t: t.flip(-1).cumsum(-1).flip(-1)  # noqa: E731
    for i, lo in enumerate(range(0, T, SPAN)):
        hi = min(T, lo + SPAN)
        run, part = back(own[:, :, lo:hi]) + ends[i + 1][..., None], back(size[:, :, lo:hi])
        whole = run[:, :, :1] + ends[i][..., None]
        out[:, :, lo:hi] = (run + (part / part[:, :, :1]).square() * whole).sqrt()
    return out


def gates_from(x, o, dv):
    """dg as the sums say, in 64 bits, from these o and dv."""
    do, v, T = x["do"].double(), x["v"].double(), x["q"].shape[2]
    at, size = (o * do).sum(-1) - (dv * v).sum(-1), ((o * do).abs() + (dv * v).abs()).sum(-1)
    ends, out = [m[0].sum((-1, -2)) for m in marks(x)], torch.zeros_like(at)
    back = lambda t: t.flip(-1).cumsum(-1).flip(-1)  # noqa: E731
    for i, lo in enumerate(range(0, T, SPAN)):
        hi = min(T, lo + SPAN)
        s, part = back(at[:, :, lo:hi]) + ends[i + 1][..., None], back(size[:, :, lo:hi])
        out[:, :, lo:hi] = s + (part / part[:, :, :1]) * (ends[i][..., None] - s[:, :, :1])
    return out
