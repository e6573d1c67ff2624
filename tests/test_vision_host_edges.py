"""More host-side checks of the vision decoder's calls (no GPU), as test_vision_host has them."""
import pytest
import torch

import s3d8_a8_linear_gb300 as s3d8
from test_vision_host import A, B, BIG, D, lib, no_device_only, two  # noqa: F401


@no_device_only
@pytest.mark.parametrize("scale", [float("nan"), float("inf"), -float("inf")])
def test_cross_attention_rejects_scales_that_are_not_finite(lib, scale):  # noqa: F811
    q, kv = two(256, 64), two(128, 64)
    assert lib.s3d8_cross_attention(A, q, B, kv, B, kv, A, 3, 5, 4, 2, 64, scale, D, None, A, BIG, None) == -1
    assert lib.s3d8_cross_attention_backward(A, q, A, q, B, kv, B, kv, A, A, A, 3, 5, 4, 2, 64, scale, D, D, D, A, BIG, None) == -1


def test_a_device_that_is_not_the_current_one_is_refused(monkeypatch):
    """Every call asks for its stream this way, before its library call."""
    monkeypatch.setattr(s3d8, "_raw_stream", lambda index: 1000 + index)
    monkeypatch.setattr(s3d8, "_current_device", lambda: 1, raising=False)
    assert s3d8._stream(torch.device("cuda", 1)) == 1001
    with pytest.raises(ValueError, match="cuda:0.*current device is cuda:1"):
        s3d8._stream(torch.device("cuda", 0))
