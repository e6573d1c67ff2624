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
