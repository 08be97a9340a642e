"""The bound by which routing proves an order in 32 bits, against its derivation: no GPU.

A softmax score is e^(x - top) / sum, made as 2^((x - top) * log2(e)) times the inverse of a sum.  In units of 2^-24 of the
row's largest score its error is at most the exponential's own (2^-22 relative: 4), its exponent's (a rounding of the
difference, one of the product, and the 24-bit constant's), the same on average over the terms of the sum, the sum's
additions, the quotient's two last places (4) and the product's rounding."""
import os
import re

import numpy as np
import pytest

from sorting_lsd_radix_gb300 import build as gbuild

LOG2E = np.float32(1.44269502162933349609375)
SOURCE = os.path.join(gbuild.CSRC, "route.cu")


def exponent_units():
    """The exponent's error over the distance, in units of 2^-24: two roundings and the constant's."""
    return 2.0 + abs(float(LOG2E) * np.log(2.0) - 1.0) * 2.0 ** 24


def average_distance(experts):
    """The largest average distance from the top under the softmax: all others at one distance d, the best d."""
    d = np.linspace(0.0, 20.0, 200_001)
    others = (experts - 1) * np.exp(-d)
    return float((others * d / (1.0 + others)).max())


def test_the_exponents_error():
    gen, worst = np.random.default_rng(5), 0.0
    for _ in range(8):
        x, top = (gen.standard_normal(1 << 18).astype(np.float32) * 10 for _ in range(2))
        top = np.maximum(x, top) + np.float32(0.5)
        distance = top.astype(np.float64) - x
        got = ((x - top) * LOG2E).astype(np.float64) * np.log(2.0)
        worst = max(worst, float((np.abs(got + distance) / distance).max()) * 2.0 ** 24)
    assert 1.5 < worst <= exponent_units()


def test_the_average_distance():
    """No random row has more than the derived one."""
    gen = np.random.default_rng(6)
    for experts in (8, 256, 1024):
        most = average_distance(experts)
        for std in (0.5, 1.0, 3.0, 10.0):
            x = gen.standard_normal((200, experts)) * std
            d = x.max(1, keepdims=True) - x
            p = np.exp(-d) / np.exp(-d).sum(1, keepdims=True)
            assert (p * d).sum(1).max() <= most
    assert 4.4 < average_distance(1024) < 4.5


@pytest.mark.parametrize("per_lane", [8, 16, 32])
def test_the_bound_covers_a_softmax_score(per_lane):
    with open(SOURCE) as f:
        rounds = int(re.search(r"score_rounds\(bool sigmoid\) \{ return sigmoid \? [0-9.]+f : \(float\)\(V \+ (\d+)\); \}", f.read())[1])
    own = 4.0 + exponent_units() / np.e
    total = 4.0 + exponent_units() * average_distance(32 * per_lane) + (per_lane - 1) + 5  # a lane's additions, the lanes'
    assert per_lane + rounds + 1 >= (own + total + 4.0 + 1.0) * (1.0 + 2.0 ** -10)
