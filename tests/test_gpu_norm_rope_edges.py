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


@pytest.mark.parametrize("T,Hq,Hk,D,rotary,inter", [(5, 7, 2, 80, 40, False), (61, 32, 8, 128, 128, False), (9, 4, 4, 256, 64, True), (40, 3, 1, 48, 6, False)])
def test_rows_whose_squares_pass_the_range_become_zeros(T, Hq, Hk, D, rotary, inter):
    """Sums of squares are fp32: past 3.4e38 the root is 0, as the header says, and with it the row,
    its gradient and its part of the weight's; no other row is touched."""
    rng, q, k, wq, wk, cos, sin, pos = _case(T, Hq, Hk, D, rotary, seed=8, fused=False)
    dz = _rand(rng, T, Hq + Hk, D)

    def run(q, k, dq, dk):
        return *s3d8.norm_rope(q, k, wq, wk, cos, sin, pos, norm.EPS, inter), s3d8.norm_rope_backward(dq, dk, q, k, wq, wk, cos, sin, pos, norm.EPS, inter)

    dq, dk = dz[:, :Hq].contiguous(), dz[:, Hq:].contiguous()
    none_q, none_k = dq.clone(), dk.clone()
    none_q[1, Hq - 1], none_k[2, 0] = 0, 0
    zq, zk, g = run(q, k, none_q, none_k)           # (no part in the weights' gradients, whatever the rows hold)
    large_q, large_k = q.clone(), k.clone()
    large_q[1, Hq - 1], large_k[2, 0] = 1e19, -3e19
    yq, yk, h = run(large_q, large_k, dq, dk)
    for got, want, at in ((yq, zq, (1, Hq - 1)), (yk, zk, (2, 0)), (h["dq"], g["dq"], (1, Hq - 1)), (h["dk"], g["dk"], (2, 0))):
        assert not got[at].any()
        want[at] = 0
        assert torch.equal(got, want)
    assert torch.equal(h["dq_norm"], g["dq_norm"]) and torch.equal(h["dk_norm"], g["dk_norm"])


@pytest.mark.parametrize("T", [5, 1700])
def test_the_append_s_rows_whose_squares_pass_the_range(T):
    rng, q, k, wq, wk, cos, sin, _ = _case(T, 8, 2, 128, 128, seed=9, fused=False)
    v = _rand(rng, T, 2, 128)
    pos, table = torch.arange(T, device=dev()).int(), torch.arange(T, device=dev()).int().view(T, 1)
    pos = pos % 16
    caches = [s3d8.KVCache.empty(T, 16, 2, 128) for _ in range(2)]
    want = s3d8.rope_append(q, k, v, cos, sin, pos, caches[0], table, q_norm=wq, k_norm=wk)
    q, k = q.clone(), k.clone()
    q[3, 1], k[2, 1] = 1e19, -3e19
    got = s3d8.rope_append(q, k, v, cos, sin, pos, caches[1], table, q_norm=wq, k_norm=wk)
    want[3, 1] = 0
    assert torch.equal(got, want)
    at = torch.arange(T, device=dev()), pos.long()
    stored, plain = caches[1].k[at], caches[0].k[at]
    plain[2, 1] = 0
    assert torch.equal(stored, plain) and torch.equal(caches[1].v[at], v)
