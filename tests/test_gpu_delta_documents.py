"""Packed documents in the gated delta rule: a reset (a log-gate of -inf) keeps apart what stands before it and behind it,
in every result and gradient, bit for bit, whatever the sizes on the other side.

What makes the results equal bit for bit: a decay over a reset is an exact zero, so that what a product takes from another
document is an exact zero, and so is what a sum adds of it.  (The other documents' gates stay as they are: a chunk's running
sum of gates, of which a decay is a difference, has other last bits with other gates before it.)  dg is held to each
document's own terms, by the bounds of test_gpu_delta.py.
"""
import math

import pytest
import torch

from test_gpu_delta import BF16, F32, call, inputs, near, on_gpu, reference, share

pytestmark = pytest.mark.gpu

TOKENS = ("q", "k", "v", "g", "beta", "do")
RESULTS = ("o", "dq", "dk", "dv", "dg", "dbeta")
# documents' first tokens: inside a chunk, at a chunk's and a mark's start, next to each other, and across marks
CUTS = [(300, (70, 150)), (300, (64, 128, 256)), (600, (1, 2, 255, 256, 257, 511)), (1100, (90, 700)), (200, (63, 199))]


def documents(seed, H, Hk, T, cuts, dk, dv, dt):
    x = inputs(seed, 1, H, Hk, T, dk, dv, dt)
    x["g"][:, :, list(cuts)] = -math.inf
    edges = (0,) + tuple(cuts) + (T,)
    return x, list(zip(edges[:-1], edges[1:]))


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("T,cuts", CUTS)
def test_documents_do_not_see_each_other(T, cuts, dt):
    x, docs = documents(T, 2, 1, T, cuts, 32, 40, dt)
    base = call(on_gpu(x))
    other = inputs(T + 1, 1, 2, 1, T, 32, 40, dt)
    for n, (lo, hi) in enumerate(docs):
        y = {name: t.clone() for name, t in x.items()}
        for name in ("q", "k", "v", "beta", "do"):
            for a, b in docs[:n] + docs[n + 1:]:
                y[name][:, :, a:b] = other[name][:, :, a:b] * (1000 if name in ("v", "do") else 1)
        if n:
            y["h0"] = y["h0"] * -7
        if n < len(docs) - 1:
            y["dhT"] = y["dhT"] * 90
        got = call(on_gpu(y))
        for name in RESULTS:
            assert torch.equal(got[name][:, :, lo:hi], base[name][:, :, lo:hi]), (name, lo, hi)
    assert torch.equal(got["h_final"], base["h_final"])  # the last document's


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("T,cuts", CUTS)
def test_a_documents_gates_are_good_to_its_own_terms(T, cuts, dt):
    # gradients of very different sizes side by side; each document against the rule over it alone
    x, docs = documents(T + 5, 2, 2, T, cuts, 24, 32, dt)
    for n, (lo, hi) in enumerate(docs):
        x["do"][:, :, lo:hi] *= 2.0 ** (-16 * (n % 2))
    x["dhT"] *= 2.0 ** (-16 * ((len(docs) - 1) % 2))
    got = call(on_gpu(x))["dg"]
    for n, (lo, hi) in enumerate(docs):
        one = {name: x[name][:, :, lo:hi] for name in TOKENS}
        one["h0"] = x["h0"] if n == 0 else None
        one["dhT"] = x["dhT"] if n == len(docs) - 1 else None
        r = reference(one)
        near("dg of %d..%d" % (lo, hi), got[:, :, lo:hi], r["dg"], share("dg", dt, F32), r["size"]["dg"])


@pytest.mark.parametrize("dt", [F32, BF16])
def test_a_document_without_a_gradient_gets_none(dt):
    # a document whose outputs take no part in the loss, between two that do
    T, cuts = 400, (90, 230)
    x, docs = documents(3, 2, 1, T, cuts, 64, 48, dt)
    x["do"][:, :, 90:230] = 0
    got = call(on_gpu(x))
    for name in ("dq", "dk", "dv", "dg", "dbeta"):
        assert torch.equal(got[name][:, :, 90:230], torch.zeros_like(got[name][:, :, 90:230])), name
