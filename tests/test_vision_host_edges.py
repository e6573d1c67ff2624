"""More host-side checks of the vision decoder's calls (no GPU), as test_vision_host has them."""
from types import SimpleNamespace

import pytest
import torch

import s3d8_a8_linear_gb300 as s3d8
from s3d8_a8_linear_gb300 import decoder
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


@pytest.mark.parametrize("which", ["q_norm", "k_norm"])
def test_norms_on_another_device_are_refused(monkeypatch, which):
    """Stand-ins for tensors, as there is one GPU at most: the append's weights have to be on its."""
    monkeypatch.setattr(decoder, "_rows", lambda t, *_: (0, (0, 0)))
    monkeypatch.setattr(decoder, "_dev", lambda *_: 0)
    monkeypatch.setattr(decoder, "_stream", lambda *_: 0)
    monkeypatch.setattr(decoder, "_load", lambda: SimpleNamespace(s3d8_norm_rope_append=lambda *_: 0))
    here, there = torch.device("cuda", 0), torch.device("cuda", 1)

    def some(*shape, device=here):
        return SimpleNamespace(shape=shape, device=device, dim=lambda: len(shape))

    def append(device):
        q, kv = some(2, 4, 64), some(2, 1, 64)
        cache = SimpleNamespace(heads=1, dim=64, k=some(1, 16, 1, 64), ref=None)
        return decoder.rope_append(q, kv, kv, some(9, 32), some(9, 32), some(2), cache, some(2, 1), q_out=q,
                                   **{which: some(64, device=device)})

    append(here)
    with pytest.raises(ValueError, match=which):
        append(there)
