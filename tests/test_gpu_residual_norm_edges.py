"""Residual norms at the ends of their range, against the formulas in 64 bits (those of
test_gpu_residual_norm, with its tolerances: 2^-8 of a bf16 output and 2^-18 of its
summands' size; (summands + 40) 2^-24 of a column sum's)."""
import numpy as np
import pytest
import torch

import s3d8_a8_linear_gb300 as s3d8
import test_gpu_residual_norm as norm
from gpu_util import dev
from test_gpu_residual_norm import BF, _f, _inputs, _lib, _rand  # noqa: F401

pytestmark = pytest.mark.gpu


def _check_backward(i, dh, dx, eps, monkeypatch):
    monkeypatch.setattr(norm, "EPS", eps)
    got = s3d8.residual_norm_backward(dh, dx, **i, eps=eps)
    ref = norm._gradients(i, _f(dh), _f(dx), 1.0, False)
    h, y, wo, wp = (_f(i[k]) for k in ("h", "y", "w_post", "w_pre"))
    inv = 1 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    a = np.abs(_f(dx) * wp)
    size = np.abs(_f(dh)) + inv * (a + np.abs(h) * inv * (a * np.abs(h) * inv).mean(-1, keepdims=True))
    rp = 1 / np.sqrt((y * y).mean(-1, keepdims=True) + eps)
    b = size * np.abs(wo)
    sizes = {"dh": size, "dy": rp * (b + np.abs(y) * rp * (b * np.abs(y) * rp).mean(-1, keepdims=True))}
    for k, t in got.items():
        if k in sizes:
            norm._close(_f(t), ref[k], tol=2.0 ** -18 * sizes[k])
        else:
            tol = (min(h.shape[0], 4096) + 40) * 2.0 ** -24 * ref["abs_" + k]
            assert (np.abs(t.double().cpu().numpy() - ref[k]) <= tol).all(), k


@pytest.mark.parametrize("M", [1, 5, 33, 700])
@pytest.mark.parametrize("D", [16, 64, 128, 256, 512, 1024, 4096, 8200])
def test_backward_without_epsilon(M, D, monkeypatch):
    """eps = 0: a group of lanes that has no row must add nothing to the columns' sums."""
    i = _inputs(M, D, True, "none", M + D)
    rng = np.random.default_rng(D)
    _check_backward(i, _rand(rng, M, D), _rand(rng, M, D), 0.0, monkeypatch)


@pytest.mark.parametrize("size", [1e-14, 1e-17])
@pytest.mark.parametrize("which", ["h", "y"])
@pytest.mark.parametrize("M,D", [(40, 64), (7, 512), (9, 1024), (5, 4096), (3, 8200)])
def test_backward_of_tiny_rows(M, D, which, size, monkeypatch):
    """Roots whose cube passes fp32's range, though no gradient does."""
    i = _inputs(M, D, True, "none", M + D)
    i[which] = (i[which].float() * size).to(BF)
    rng = np.random.default_rng(D)
    _check_backward(i, _rand(rng, M, D), _rand(rng, M, D), 0.0, monkeypatch)


@pytest.mark.parametrize("M,D", [(2, 64), (5, 512), (3, 1024), (3, 4096), (400, 2048), (310, 8192), (3, 16384)])
def test_rows_whose_squares_pass_the_range_become_zeros(M, D):
    """Sums of squares are fp32: past 3.4e38 the root is 0, as the header says, and no other row is touched."""
    i = _inputs(M, D, True, "none", D)
    plain = [t.clone() for t in s3d8.residual_norm(**i)] + [t.clone() for t in s3d8.residual_norm_quant(**i)[1:]]
    i["y"][1] = 1e19
    h, x = s3d8.residual_norm(**i)
    _, q, s = s3d8.residual_norm_quant(**i)
    assert torch.equal(h[1], i["h"][1])                     # the update is 0, the stream stays
    norm._close(_f(x[1:2]), norm._norm(_f(i["h"][1:2]), _f(i["w_pre"])))
    i["h"][1] = -3e19
    h, x = s3d8.residual_norm(**i)
    _, q, s = s3d8.residual_norm_quant(**i)
    assert torch.equal(h[1], i["h"][1]) and bool((x[1] == 0).all()) and bool((q[1] == 0).all()) and float(s[1]) == 0.0
    keep = [m for m in range(M) if m != 1]
    for got, want in zip((h, x, q, s), plain):
        assert torch.equal(got[keep], want[keep])


def test_a_second_derivative_is_refused():
    """The gradients are kernels without a graph: a loss that differentiates through them raises instead of losing terms."""
    i = _inputs(3, 64, True, "scalar", 1)
    leaf = {k: t.clone().requires_grad_() for k, t in i.items()}
    _, x = s3d8.ResidualNorm.apply(leaf["h"], leaf["y"], leaf["w_post"], leaf["gate"], leaf["w_pre"], 1.0, 1e-5, True)
    (first,) = torch.autograd.grad(x.float().square().sum(), leaf["h"], create_graph=True)
    with pytest.raises(RuntimeError, match="twice"):
        (first.float().square().sum() + leaf["h"].float().square().sum()).backward()
