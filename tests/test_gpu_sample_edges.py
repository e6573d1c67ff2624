"""The next token at the ends of fp32's range (against the definition of test_gpu_sample)."""
import numpy as np
import pytest
import torch

from gpu_util import dev
from test_gpu_sample import BF, _check, _lib  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 24, 256, 8200])
@pytest.mark.parametrize("value,temp", [(float("inf"), 1.0), (2.0, 1e-20), (-2.0, 1e-20), (3.0, 1e-38), (-3.0, 1e-38), (5.0, 1e-45), (0.0, 1e-45)])
def test_rows_that_are_all_counted(V, value, temp):
    """Equal logits, infinite or over a temperature that takes them past fp32's range, alone and
    with lower ones that have no weight: a lane without any of those and one that has nothing but
    padding take no weight from each other."""
    x = torch.full((3, V), value, dtype=BF, device=dev())
    if V > 2:
        x[1, 1::2] = value - 1.0 if np.isfinite(value) else 7.0
        x[2, V // 2:] = -float("inf")
    for u in (0.0, 2.0 ** -17, 0.3, 1.0 - 2.0 ** -24):
        _check(x, u, temp)
        _check(x, u, temp, p=0.5)


@pytest.mark.parametrize("temp", [1e36, 3e37, 2e38])
def test_temperatures_near_the_largest_number(temp):
    """Logits a few temperatures apart, which fill the range, and ones that are never drawn."""
    low = torch.finfo(BF).min
    x = torch.tensor([3e38, low, 0.0, 1e38, -1e38, -float("inf"), float("nan"), 1.0, low, -2e38, 2.5e38], dtype=BF, device=dev())
    x = torch.cat((x, torch.full((3000,), -float("inf"), dtype=BF, device=dev()))).expand(6, -1)
    _check(x, np.array([0.0, 0.2, 0.4, 0.6, 0.8, 0.999]), temp)


@pytest.mark.parametrize("temp", [2.0 ** -79, 2.0 ** -81, 2.0 ** -110, 2.0 ** -126])
def test_temperatures_near_the_smallest_number(temp):
    """Logits a few temperatures apart: neither 1 / T nor a logit over T is infinite."""
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.standard_normal((6, 3000)) * 8.0 * temp).to(BF).to(dev())
    _check(x, np.array([0.0, 0.2, 0.4, 0.6, 0.8, 0.999]), temp)
    x[:, 7] = 1.0
    assert int(_check(x, 0.5, temp)[0]) == 7
