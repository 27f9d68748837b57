"""Backward of attention to another sequence's keys against differences of the loss (cross_differences.py)."""
import pytest
import torch

from cross_differences import NAMES, Differences
from gpu_util import ensure_built, f64
from test_cross_differences import CASES
from test_gpu_cross import step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


@pytest.mark.parametrize("sizes", CASES + [(1, 1, 2, 1, 3, 700, 64, [611]), (1, 1, 1, 1, 150, 20, 128, [17])])
def test_backward_along_the_gradient(sizes):
    q, k, v, do, _, _, grads, scale = step(*sizes, seed=9, poison=False)
    D = Differences(*(f64(t) for t in (q, k, v, do)), sizes[-1], scale)
    for i, name in enumerate(NAMES):
        assert torch.isfinite(grads[i]).all()
        assert D.off(i, f64(grads[i])) <= 1, (name, D.off(i, f64(grads[i])))
