"""A seeded random sweep of the gated delta rule and of layer norm against the float64 code and the error bounds of
test_gpu_delta.py.

Drawn ranges:
- the rule, forward and backward: B <= 4, up to 160 heads a batch, T <= 1100, dk <= 128, dv <= 320 (both ways to give
  columns to a workgroup, whole and in segments), every type and gate recipe, keys shared by value heads, with and
  without lengths and resets;
- single tokens: B <= 6, H <= 6, n <= 5, dk <= 256, dv <= 300, every type;
- layer norm, forward and backward: B <= 4, T <= 300, D <= 16384, every type pair.

It runs 45 configurations by default (15 of each).  GLA_SWEEP_DELTA=500 runs that many of each, GLA_SWEEP_SEED draws
another sample.
"""
import os
import random

import pytest
import torch

from test_gpu_delta import BF16, F32, check, inputs, test_delta_step as run_step, test_layernorm as run_norm

pytestmark = pytest.mark.gpu

N = int(os.environ.get("GLA_SWEEP_DELTA", "15"))
SEED = int(os.environ.get("GLA_SWEEP_SEED", "4242"))


def _log(rng, hi):
    """1 .. hi, spread over the logarithm."""
    return max(1, min(hi, int(round(2 ** rng.uniform(0, hi.bit_length())))))


def rule_case(rng):
    dk, dv = rng.choice([16, 64, 100, 128, _log(rng, 128)]), rng.choice([32, 64, 80, 128, _log(rng, 320)])
    B, Hk, G = rng.randint(1, 4), rng.choice([1, 2, 3, _log(rng, 40)]), rng.choice([1, 1, 2, 4])
    T = rng.choice([rng.randint(1, 70), rng.randint(60, 400), rng.randint(300, 1100)])
    while B * Hk * G * T * dk * dv > 3e8:  # (the plain code's time)
        B, Hk, T = max(1, B - 1), max(1, Hk // 2), max(1, T * 2 // 3)
    lens = [rng.randint(0, T) for _ in range(B)] if rng.random() < 0.4 else None
    return (rng.randrange(1 << 30), B, Hk * G, Hk, T, dk, dv, rng.choice([F32, BF16]),
            rng.choice(["mid", "weak", "strong", "zero", "mixed"]), rng.choice([0, 0, 3]), lens)


def step_case(rng):
    Hk, G = rng.randint(1, 3), rng.randint(1, 2)
    return (rng.randint(1, 6), Hk * G, Hk, rng.choice([1, 1, 2, 5]), rng.randint(1, 256), rng.randint(1, 300), rng.choice([F32, BF16]))


def norm_case(rng):
    D = rng.choice([rng.randint(1, 600), _log(rng, 16384), 8 * _log(rng, 2048)])
    return (rng.randint(1, 4), rng.randint(1, max(1, min(300, 400000 // D))), D) + rng.choice([(F32, F32), (BF16, BF16), (BF16, F32)])


def cases(draw, salt):
    rng = random.Random(SEED + salt)
    return [draw(rng) for _ in range(N)]


# many heads, 128 columns a workgroup: whole, and in segments; and the widest values
FULL = [(1, 1, 140, 70, 70, 64, 100, BF16, "mid", 0, None), (2, 2, 70, 70, 100, 40, 72, F32, "mid", 0, [100, 3]),
        (3, 2, 10, 5, 640, 64, 80, BF16, "weak", 3, [640, 391]), (4, 1, 24, 24, 700, 32, 70, F32, "weak", 0, None),
        (5, 1, 2, 1, 130, 16, 1024, BF16, "mid", 0, None)]


@pytest.mark.parametrize("case", FULL + cases(rule_case, 1), ids=str)
def test_random_rule(case):
    seed, B, H, Hk, T, dk, dv, dt, gates, resets, lens = case
    check(inputs(seed, B, H, Hk, T, dk, dv, dt, gates, resets), None if lens is None else torch.tensor(lens), "sweep")


@pytest.mark.parametrize("case", cases(step_case, 2), ids=str)
def test_random_single_tokens(case):
    run_step(*case)


@pytest.mark.parametrize("case", cases(norm_case, 3), ids=str)
def test_random_norm(case):
    run_norm(*case)
