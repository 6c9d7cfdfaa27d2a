"""A seeded random sweep of the recurrent-block operators against the float64 code and the error bounds of
test_gpu_block.py, element by element.

Drawn ranges:
- recurrence, forward and backward: B <= 5, T <= 1400, D <= 1000, every type, mode and gate recipe, with and
  without lengths and resets;
- join, forward and backward: every H <= 2048 and d with H d <= 8192 (narrow heads by the hundred, wide ones,
  widths that are no multiple of 8), B <= 4, T <= 60, every type pair, each part present three times in four;
- gla_step: B <= 6, H <= 4, n <= 5, dk <= 256, dv <= 300, every type.

It runs 60 configurations by default (20 of each).  GLA_SWEEP_BLOCK=2000 runs that many of each,
GLA_SWEEP_SEED draws another sample.
"""
import os
import random

import pytest
import torch

from test_gpu_block import (BF16, F32, check_join, check_recur, join_inputs, recur_inputs, test_step as run_step)

pytestmark = pytest.mark.gpu

N = int(os.environ.get("GLA_SWEEP_BLOCK", "20"))
SEED = int(os.environ.get("GLA_SWEEP_SEED", "4242"))


def _log(rng, hi):
    """1 .. hi, spread over the logarithm."""
    return max(1, min(hi, int(round(2 ** rng.uniform(0, hi.bit_length())))))


def recur_case(rng):
    B, D = rng.randint(1, 5), rng.choice([1, 7, 64, 65, 130, 900, _log(rng, 1000)])
    T = rng.choice([rng.randint(1, 40), rng.randint(1, 300), rng.randint(200, 1400)])
    lens = [rng.randint(0, T) for _ in range(B)] if rng.random() < 0.4 else None
    return (rng.randrange(1 << 30), B, T, D, rng.choice([F32, BF16]), rng.choice(["plain", "lerp", "norm"]),
            rng.choice(["mid", "weak", "strong", "zero"]), rng.choice([0, 0, 3]), lens)


def join_case(rng):
    if rng.random() < 0.5:  # by heads first: many narrow ones
        H = _log(rng, 2048)
        d = _log(rng, 8192 // H)
    else:
        d = _log(rng, 8192)
        H = _log(rng, min(2048, 8192 // d))
    if rng.random() < 0.4 and d >= 8:
        d -= d % 8
    T = rng.randint(1, max(1, min(60, 60000 // (H * d))))
    parts = {p: rng.random() < 0.75 for p in ("post", "gate", "residual", "scale", "pre")}
    return (rng.randrange(1 << 30), rng.randint(1, 4), H, T, d, rng.choice([(F32, F32), (BF16, BF16), (BF16, F32)]),
            rng.choice(["silu", "sigmoid"]), parts, rng.choice(["both", "both", "d_out", "d_normed"]))


def step_case(rng):
    return (rng.randint(1, 6), rng.randint(1, 4), rng.choice([1, 1, 2, 5]), rng.randint(1, 256), rng.randint(1, 300),
            rng.choice([F32, BF16]))


def cases(draw, salt):
    rng = random.Random(SEED + salt)
    return [draw(rng) for _ in range(N)]


@pytest.mark.parametrize("case", cases(recur_case, 1), ids=str)
def test_random_recurrence(case):
    seed, B, T, D, dt, mode, gates, resets, lens = case
    x, g, dh, h0, dhT = recur_inputs(seed, B, T, D, dt, gates, resets)
    check_recur(x, g, dh, h0, dhT, None if lens is None else torch.tensor(lens), mode, "sweep")


@pytest.mark.parametrize("case", cases(join_case, 2), ids=str)
def test_random_join(case):
    seed, B, H, T, d, (dt, st), act, parts, grads = case
    y, a, d_out, d_normed = join_inputs(seed, B, H, T, d, dt, st, **parts)
    if not parts["pre"] or grads == "d_out":
        d_normed = None
    if d_normed is not None and grads == "d_normed":
        d_out = None
    check_join(y, a, d_out, d_normed, act, "sweep")


@pytest.mark.parametrize("case", cases(step_case, 3), ids=str)
def test_random_step(case):
    run_step(*case)
