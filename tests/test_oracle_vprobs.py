"""Pins of the probability-verify and 8-bit projection references on the pages'
own numbers and on exact laws (CPU)."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import int8 as oi
from oracle import vprobs as ov


def test_the_worked_three_token_example():
    """[P4 "Speculative decoding"] p = (0.2, 0.5, 0.3), q = (0.5, 0.3, 0.2): token 0
    is kept with 0.4, tokens 1 and 2 always; the residual is (0, 2/3, 1/3)."""
    p = np.array([[0.2, 0.5, 0.3], [0.0, 0.0, 1.0]])
    q = np.array([[0.5, 0.3, 0.2]])
    for x, u, kept in ((0, 0.39, 1), (0, 0.41, 0), (1, 0.999, 1), (2, 0.999, 1)):
        assert ov.verify_probs_row(p, q, [x], 1, [u], 0.5).accepted == kept
    for v, token in ((0.0, 1), (0.66, 1), (0.67, 2), (0.999, 2)):
        r = ov.verify_probs_row(p, q, [0], 1, [0.9], v)
        assert list(r.tokens) == [token, -1]


def test_the_output_is_distributed_as_the_target():
    """Integrating the rule over its uniforms gives p exactly (eq. 39.4's
    identity), here on a grid fine enough to count."""
    p, q = np.array([0.25, 0.5, 0.125, 0.125]), np.array([0.5, 0.25, 0.25, 0.0])
    n = 64
    mass = np.zeros(4)
    grid = (np.arange(n) + 0.5) / n
    for x in range(3):
        for u in grid:
            for v in grid:
                r = ov.verify_probs_row(np.stack([p, p]), q[None], [x], 1, [u], v)
                mass[r.tokens[0]] += q[x] / n / n
    assert np.abs(mass - p).max() < 2.0 / n


def test_certain_proposals_keep_the_target_too():
    p = np.array([0.5, 0.25, 0.25])
    n = 64
    grid = (np.arange(n) + 0.5) / n
    mass = np.zeros(3)
    for u in grid:
        for v in grid:
            mass[ov.verify_probs_row(np.stack([p, p]), None, [1], 1, [u], v).tokens[0]] += 1 / n / n
    assert np.abs(mass - p).max() < 2.0 / n


@pytest.mark.parametrize("seed", range(4))
def test_codes_are_the_nearest_whole_numbers(seed):
    """Against rational arithmetic: round half to even of the exact quotient."""
    rng = np.random.default_rng(seed)
    x = rng.normal(0, 1, (4, 64)).astype(np.float32)
    x[1] = np.round(x[1] * 8) / 8                  # many exact halves
    x[1, 0] = 127.0
    x[2] *= np.float32(1e-39)                      # scales below the normal range
    x[3] = 0
    codes, scale = oi.quantize_rows(x)
    assert scale[3] == 0 and not codes[3].any()
    for r in range(3):
        s = Fraction(float(scale[r]))
        for v, c in zip(x[r], codes[r]):
            want = max(-127, min(127, round(Fraction(float(v)) / s)))   # round(): ties to even
            assert c == want
