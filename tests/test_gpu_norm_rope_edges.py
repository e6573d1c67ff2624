"""Normed rotary heads at the ends of fp32's range, against the formulas in 64 bits (those of
test_gpu_norm_rope, with its tolerances)."""
import pytest
import torch

import s3d8_a8_linear_gb300 as s3d8
import test_gpu_norm_rope as norm
from gpu_util import dev
from test_gpu_norm_rope import BF, _backward, _case, _close, _close_sum, _forward, _lib, _rand  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", [1e-14, 1e-17, 4e-20])
@pytest.mark.parametrize("T,Hq,Hk,D,rotary,inter", [(5, 7, 2, 80, 40, False), (61, 32, 8, 128, 128, False), (9, 4, 4, 256, 64, True)])
def test_tiny_rows_without_epsilon(T, Hq, Hk, D, rotary, inter, size, monkeypatch):
    """Roots whose square passes fp32's range, though no gradient does.  (Squares of 4e-20 are
    subnormal, 2^-149 apart: their mean is right to 2^-20 and its root to 2^-21, which is within
    the outputs' tolerance of 2^-16, and within a quarter of a column sum's: of 10 rows or more,
    50 2^-24 / 4.)"""
    monkeypatch.setattr(norm, "EPS", 0.0)
    rng, q, k, wq, wk, cos, sin, pos = _case(T, Hq, Hk, D, rotary, seed=7)
    q, k = (q.float() * size).to(BF), (k.float() * size).to(BF)
    zq, zk = s3d8.norm_rope(q, k, wq, wk, cos, sin, pos, 0.0, inter)
    _close(zq, *_forward(q, wq, cos, sin, pos, inter))
    _close(zk, *_forward(k, wk, cos, sin, pos, inter))
    dz = _rand(rng, T, Hq + Hk, D)
    dq, dk = dz[:, :Hq], dz[:, Hq:]
    g = s3d8.norm_rope_backward(dq, dk, q, k, wq, wk, cos, sin, pos, 0.0, inter)
    for dz_, x, w, dx, dw in ((dq, q, wq, "dq", "dq_norm"), (dk, k, wk, "dk", "dk_norm")):
        ref, scale, dw_ref, dw_size = _backward(dz_, x, w, cos, sin, pos, inter)
        _close(g[dx], ref, scale)
        _close_sum(g[dw], dw_ref, 1.25 * dw_size, T * x.shape[1])
