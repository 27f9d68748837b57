"""That the check of gradients against differences (cross_differences.py) takes right ones and no others (no GPU)."""
import numpy as np
import pytest

from cross_differences import NAMES, Differences
from plain64 import bf16_round

CASES = [(2, 1, 2, 1, 6, 40, 64, [33]), (2, 2, 2, 2, 20, 60, 128, [20, 60]), (4, 2, 4, 2, 3, 30, 64, [30, 7])]


def case(B, B_kv, H, H_kv, N_q, N_kv, d, lengths, seed=1):
    rng = np.random.default_rng(seed)
    q, do = (bf16_round(rng.standard_normal((B, H, N_q, d))) for _ in range(2))
    k, v = (bf16_round(rng.standard_normal((B_kv, H_kv, N_kv, d))) for _ in range(2))
    return Differences(q, k, v, do, lengths, d ** -0.5)


WRONG = {
    "negated": lambda g: -g,
    "halved": lambda g: g / 2,
    "of 3 / 4": lambda g: 0.75 * g,
    "half as much again": lambda g: 1.5 * g,
    "eight times": lambda g: 8 * g,
    "rows permuted": lambda g: g[:, :, np.random.default_rng(5).permutation(g.shape[2])],
    "a column further": lambda g: np.roll(g, 1, 3),
    "of another head": lambda g: np.roll(g, 1, 1) if g.shape[1] > 1 else np.roll(g, 1, 2),
    "zeros": np.zeros_like,
}


@pytest.mark.parametrize("sizes", CASES)
def test_the_formula_agrees_with_differences(sizes):
    D = case(*sizes)
    for i, name in enumerate(NAMES):
        assert abs((D.ref[i] * D.directions[i]).sum() - D.slopes[i]) <= 1e-6 * abs(D.slopes[i]), name
        assert D.off(i, bf16_round(D.ref[i])) <= 1, name


@pytest.mark.parametrize("wrong", WRONG)
@pytest.mark.parametrize("sizes", CASES)
def test_a_wrong_gradient_is_seen(sizes, wrong):
    D = case(*sizes)
    for i, name in enumerate(NAMES):
        assert D.off(i, WRONG[wrong](D.ref[i])) > 1, name
