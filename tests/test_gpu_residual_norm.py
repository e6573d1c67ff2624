"""Residual norms against their formulas in 64 bits, and their gradients against
the formulas' and against differences.

Tolerances.  A bf16 output is off by its rounding, at most 2^-9 of its size, and
by the fp32 arithmetic in front of it: a handful of operations at 2^-24 each of
the summands' size, below 2^-18 here.  2^-8 |ref| + 1e-5 covers both (the summands
are of order 1).  An fp32 column sum over m rows is off by at most (m + 20) 2^-24
of the sum of its summands' sizes, those inside of G among them.
"""
import numpy as np
import pytest
import torch

import s3d8_a8_linear_gb300 as s3d8
from gpu_util import bf16_to_f64, dev, guarded

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    s3d8.load(build_if_missing=True)
    torch.cuda.set_device(0)
    yield
    assert s3d8.device_status() == 0


def _rand(rng, *shape, scale=1.0, mean=0.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale + mean).astype(np.float32)).to(BF).to(dev())


def _inputs(M, D, post, gate, seed):
    rng = np.random.default_rng(seed)
    return dict(h=_rand(rng, M, D), y=_rand(rng, M, D, scale=0.5),
                w_post=_rand(rng, D, scale=0.1, mean=1.0) if post else None,
                gate={"none": None, "scalar": _rand(rng, 1), "channel": _rand(rng, D)}[gate],
                w_pre=_rand(rng, D, scale=0.1, mean=1.0))


def _f(t):
    return None if t is None else bf16_to_f64(t)


def _gain(gate, alpha, tanh):
    g = np.ones(1) if gate is None else gate
    return alpha * (np.tanh(g) if tanh else g)


def _update(h, y, w_post, gate, alpha, tanh):
    """h' before its rounding, in 64 bits."""
    u = y
    if w_post is not None:
        u = y / np.sqrt((y * y).mean(-1, keepdims=True) + EPS) * w_post
    return h + _gain(gate, alpha, tanh) * u


def _norm(h, w):
    return h / np.sqrt((h * h).mean(-1, keepdims=True) + EPS) * w


def _close(got, ref, rel=2.0 ** -8, tol=1e-5):
    excess = np.abs(got - ref) - (rel * np.abs(ref) + tol)
    assert (excess <= 0).all(), f"off by {excess.max()} beyond the tolerance"


SIZES = [(1, 8), (1, 4096), (3, 16), (5, 256), (7, 264), (2, 1000), (33, 4096), (4, 8192), (3, 8200),
         (2, 14336), (3, 16384), (700, 64), (401, 528)]
FORMS = [(True, "none", 1.0, False), (False, "none", 0.22, False), (True, "scalar", 1.0, True),
         (False, "scalar", 2.5, False), (True, "channel", 0.22, False), (False, "channel", 1.0, True)]


@pytest.mark.parametrize("post,gate,alpha,tanh", FORMS)
@pytest.mark.parametrize("M,D", SIZES)
def test_forward(M, D, post, gate, alpha, tanh):
    i = _inputs(M, D, post, gate, M * 31 + D)
    out, check_h = guarded((M, D), BF, 3.0)
    x, check_x = guarded((M, D), BF, 3.0)
    got_h, got_x = s3d8.residual_norm(**i, alpha=alpha, eps=EPS, tanh_gate=tanh, h_out=out, x=x)
    torch.cuda.synchronize()
    check_h(), check_x()
    _close(_f(got_h), _update(_f(i["h"]), _f(i["y"]), _f(i["w_post"]), _f(i["gate"]), alpha, tanh))
    _close(_f(got_x), _norm(_f(got_h), _f(i["w_pre"])))


@pytest.mark.parametrize("M,D", [(1, 16), (1, 4096), (5, 8192), (37, 4096), (3, 14336), (300, 272)])
def test_codes_are_those_of_quantize_act(M, D):
    i = _inputs(M, D, True, "scalar", D)
    h, x = s3d8.residual_norm(**i, tanh_gate=True)
    want_q, want_s = s3d8.quantize_act(x)
    hq, q, s = s3d8.residual_norm_quant(**i, tanh_gate=True)
    torch.cuda.synchronize()
    assert torch.equal(hq, h) and torch.equal(q, want_q) and torch.equal(s, want_s)


def test_parts_alone_and_in_place():
    M, D = 19, 1024
    i = _inputs(M, D, True, "none", 4)
    same, x = s3d8.residual_norm(i["h"], w_pre=i["w_pre"])
    assert same is i["h"]
    _close(_f(x), _norm(_f(i["h"]), _f(i["w_pre"])))
    h, none = s3d8.residual_norm(i["h"], i["y"], i["w_post"])
    assert none is None
    _close(_f(h), _update(_f(i["h"]), _f(i["y"]), _f(i["w_post"]), None, 1.0, False))
    stream = i["h"].clone()
    h2, x2 = s3d8.residual_norm(stream, i["y"], i["w_post"], w_pre=i["w_pre"], h_out=stream)
    assert h2 is stream and torch.equal(stream, h)
    _close(_f(x2), _norm(_f(h), _f(i["w_pre"])))
    empty = torch.empty((0, D), dtype=BF, device=dev())
    h3, x3 = s3d8.residual_norm(empty, empty, w_pre=i["w_pre"])
    assert h3.shape == x3.shape == (0, D)


# more rows than the GPU takes at once: several a CTA, at every width's number of threads and stages
MANY = [(310, 1032), (1500, 2048), (307, 2056), (700, 4096), (320, 8192), (311, 8200), (309, 16384), (5000, 512), (9000, 128),
        (20000, 8), (3001, 1024)]


@pytest.mark.parametrize("post,gate,alpha,tanh", [FORMS[0], FORMS[3], FORMS[4]])
@pytest.mark.parametrize("M,D", MANY)
def test_many_rows(M, D, post, gate, alpha, tanh):
    i = _inputs(M, D, post, gate, M + D)
    rng = np.random.default_rng(D)
    dh, dx = _rand(rng, M, D), _rand(rng, M, D)
    h, x = s3d8.residual_norm(**i, alpha=alpha, eps=EPS, tanh_gate=tanh)
    _close(_f(h), _update(_f(i["h"]), _f(i["y"]), _f(i["w_post"]), _f(i["gate"]), alpha, tanh))
    _close(_f(x), _norm(_f(h), _f(i["w_pre"])))
    if D % 16 == 0:
        hq, q, s = s3d8.residual_norm_quant(**i, alpha=alpha, eps=EPS, tanh_gate=tanh)
        want_q, want_s = s3d8.quantize_act(x)
        assert torch.equal(hq, h) and torch.equal(q, want_q) and torch.equal(s, want_s)
    same, alone = s3d8.residual_norm(h, w_pre=i["w_pre"])
    assert same is h and torch.equal(alone, x)
    assert torch.equal(s3d8.residual_norm(**{**i, "w_pre": None}, alpha=alpha, eps=EPS, tanh_gate=tanh)[0], h)
    got = s3d8.residual_norm_backward(dh, dx, **i, alpha=alpha, eps=EPS, tanh_gate=tanh)
    again = s3d8.residual_norm_backward(dh, dx, **i, alpha=alpha, eps=EPS, tanh_gate=tanh)
    ref = _gradients(i, _f(dh), _f(dx), alpha, tanh)
    for k, t in got.items():
        assert torch.equal(t, again[k]), k
        if k in ("dh", "dy"):
            _close(_f(t), ref[k])
        else:
            summands = M * (D if t.numel() == 1 and D > 1 else 1)
            tol = (min(summands, 4096) + 40) * 2.0 ** -24 * ref["abs_" + k]
            assert (np.abs(t.double().cpu().numpy() - ref[k]) <= tol + 1e-30).all(), k


@pytest.mark.parametrize("M,D", [(40, 64), (700, 1024), (350, 4096), (6, 8192), (200, 8200)])
def test_absent_gradients_at_every_form(M, D):
    """dh, dx or both missing, with and without a block's output."""
    i = _inputs(M, D, True, "scalar", M)
    rng = np.random.default_rng(D)
    dh, dx = _rand(rng, M, D), _rand(rng, M, D)
    zero = np.zeros((M, D))
    for a, b in ((dh, None), (None, dx), (None, None)):
        fa, fb = zero if a is None else _f(a), zero if b is None else _f(b)
        got = s3d8.residual_norm_backward(a, b, **i, tanh_gate=True)
        ref = _gradients(i, fa, fb, 1.0, True)
        _close(_f(got["dh"]), ref["dh"])
        _close(_f(got["dy"]), ref["dy"])
        alone = s3d8.residual_norm_backward(a, b, i["h"], w_pre=i["w_pre"])
        assert set(alone) == {"dh", "dw_pre"} and torch.equal(alone["dh"], got["dh"])
        assert torch.equal(alone["dw_pre"], got["dw_pre"])


def test_zero_rows_and_extreme_sizes():
    D = 512
    h = torch.zeros((3, D), dtype=BF, device=dev())
    y = torch.zeros_like(h)
    y[1] = 1e18      # its square passes fp32's range in the sum
    y[2] = 1e-18
    w = torch.ones(D, dtype=BF, device=dev())
    out, x = s3d8.residual_norm(h, y, w, w_pre=w)
    q = s3d8.residual_norm_quant(h, y, w, w_pre=w)
    torch.cuda.synchronize()
    assert bool((out[0] == 0).all()) and bool((x[0] == 0).all())
    assert bool((q[1][0] == 0).all()) and float(q[2][0]) == 0.0
    _close(_f(out[2]), _update(_f(h[2:]), _f(y[2:]), _f(w), None, 1.0, False)[0])


def _gradients(i, dh, dx, alpha, tanh):
    """The formulas in 64 bits; with each, the sum of its summands' sizes."""
    h, y, wo, g, wp = (_f(i[k]) for k in ("h", "y", "w_post", "gate", "w_pre"))
    inv = 1 / np.sqrt((h * h).mean(-1, keepdims=True) + EPS)
    hat, a = h * inv, dx * wp
    G = dh + inv * (a - hat * (a * hat).mean(-1, keepdims=True))
    size = np.abs(dh) + inv * (np.abs(a) + np.abs(hat) * np.abs(a * hat).mean(-1, keepdims=True))   # of G's summands
    gain = _gain(g, alpha, tanh)
    r = 1 / np.sqrt((y * y).mean(-1, keepdims=True) + EPS) if wo is not None else 1.0
    unit, du = y * r, G * gain
    b = du * (1.0 if wo is None else wo)
    dy = r * (b - unit * (b * unit).mean(-1, keepdims=True)) if wo is not None else du
    got = {"dh": G, "dy": dy, "dw_pre": (dx * hat).sum(0), "abs_dw_pre": np.abs(dx * hat).sum(0)}
    if wo is not None:
        got["dw_post"], got["abs_dw_post"] = (du * unit).sum(0), np.abs(size * gain * unit).sum(0)
    if g is not None:
        slope = alpha * ((1 - np.tanh(g) ** 2) if tanh else np.ones_like(g))
        t = G * unit * (1.0 if wo is None else wo)
        got["dgate"], got["abs_dgate"] = slope * t.sum(0), np.abs(slope) * np.abs(
            size * unit * (1.0 if wo is None else wo)).sum(0)
        if g.size == 1:
            got["dgate"], got["abs_dgate"] = got["dgate"].sum(keepdims=True), got["abs_dgate"].sum(keepdims=True)
    return got


@pytest.mark.parametrize("post,gate,alpha,tanh", FORMS)
@pytest.mark.parametrize("M,D", SIZES)
def test_backward(M, D, post, gate, alpha, tanh):
    i = _inputs(M, D, post, gate, M * 37 + D)
    rng = np.random.default_rng(D)
    dh, dx = _rand(rng, M, D), _rand(rng, M, D)
    got = s3d8.residual_norm_backward(dh, dx, **i, alpha=alpha, eps=EPS, tanh_gate=tanh)
    again = s3d8.residual_norm_backward(dh, dx, **i, alpha=alpha, eps=EPS, tanh_gate=tanh)
    torch.cuda.synchronize()
    ref = _gradients(i, _f(dh), _f(dx), alpha, tanh)
    assert set(got) == {k for k in ref if not k.startswith("abs")}
    for k, t in got.items():
        assert torch.equal(t, again[k]), f"{k} differs from call to call"
        if k in ("dh", "dy"):
            _close(_f(t), ref[k])
        else:
            summands = M * (D if t.numel() == 1 and D > 1 else 1)
            tol = (min(summands, 4096) + 40) * 2.0 ** -24 * ref["abs_" + k]
            assert (np.abs(t.double().cpu().numpy() - ref[k]) <= tol + 1e-30).all(), k


@pytest.mark.parametrize("post,gate,alpha,tanh", FORMS)
def test_backward_against_differences(post, gate, alpha, tanh):
    """Central differences of the formulas in 64 bits along random directions."""
    M, D = 4, 64
    i = _inputs(M, D, post, gate, 11)
    rng = np.random.default_rng(12)
    dh, dx = _rand(rng, M, D), _rand(rng, M, D)
    base = {k: _f(t) for k, t in i.items()}

    def stream(**c):     # the backward call takes h' as stored: the point of differentiation
        c = {**base, **c}
        return _update(c["h"], c["y"], c["w_post"], c["gate"], alpha, tanh), c["w_pre"]

    # choose the forward call's h such that h' is exactly the stored tensor
    base["h"] = base["h"] - _update(np.zeros((M, D)), base["y"], base["w_post"], base["gate"], alpha, tanh)

    def loss(**c):
        hp, w = stream(**c)
        return (_f(dh) * hp).sum() + (_f(dx) * _norm(hp, w)).sum()

    got = s3d8.residual_norm_backward(dh, dx, **i, alpha=alpha, eps=EPS, tanh_gate=tanh)
    names = {"h": "dh", "y": "dy", "w_post": "dw_post", "gate": "dgate", "w_pre": "dw_pre"}
    for k, g in names.items():
        if base[k] is None:
            continue
        grad = got[g].double().cpu().numpy()
        for _ in range(3):
            d = rng.standard_normal(base[k].shape)
            e = 1e-5
            diff = (loss(**{k: base[k] + e * d}) - loss(**{k: base[k] - e * d})) / (2 * e)
            # bf16 gradients: 2^-9 each; the difference itself: e^2 and 2^-52 / e
            assert abs((grad * d).sum() - diff) <= 2.0 ** -8 * np.abs(grad * d).sum() + 1e-5, k


def test_missing_gradients_and_autograd():
    M, D = 6, 320
    i = _inputs(M, D, True, "scalar", 3)
    rng = np.random.default_rng(8)
    dh, dx = _rand(rng, M, D), _rand(rng, M, D)
    zero = np.zeros((M, D))
    for a, b in ((dh, None), (None, dx), (None, None)):
        got = s3d8.residual_norm_backward(a, b, **i, tanh_gate=True)
        ref = _gradients(i, zero if a is None else _f(a), zero if b is None else _f(b), 1.0, True)
        _close(_f(got["dh"]), ref["dh"])
        _close(_f(got["dy"]), ref["dy"])
    leaf = {k: t.clone().requires_grad_() for k, t in i.items()}
    h2, x = s3d8.ResidualNorm.apply(leaf["h"], leaf["y"], leaf["w_post"], leaf["gate"], leaf["w_pre"], 1.0, EPS, True)
    torch.autograd.backward((h2, x), (dh, dx))
    want = s3d8.residual_norm_backward(dh, dx, **{**i, "h": h2.detach()}, tanh_gate=True)
    assert torch.equal(leaf["h"].grad, want["dh"]) and torch.equal(leaf["y"].grad, want["dy"])
    for k, g in (("w_post", "dw_post"), ("gate", "dgate"), ("w_pre", "dw_pre")):
        assert torch.equal(leaf[k].grad, want[g].to(BF)), k
    # a norm alone, of which only x is used further on
    h = i["h"].clone().requires_grad_()
    _, x = s3d8.ResidualNorm.apply(h, None, None, None, i["w_pre"])
    x.backward(dx)
    want = s3d8.residual_norm_backward(None, dx, i["h"], w_pre=i["w_pre"])
    assert torch.equal(h.grad, want["dh"])
    none = s3d8.residual_norm_backward(dh[:0], dx[:0], **{**i, "h": i["h"][:0], "y": i["y"][:0]})
    assert all(bool((none[k] == 0).all()) for k in ("dw_pre", "dw_post", "dgate"))


def test_refusals():
    i = _inputs(2, 64, True, "none", 1)
    with pytest.raises(ValueError):
        s3d8.residual_norm(i["h"], i["y"][:1], w_pre=i["w_pre"])
    with pytest.raises(TypeError):
        s3d8.residual_norm(i["h"].float(), i["y"], w_pre=i["w_pre"])
    with pytest.raises(ValueError):
        s3d8.residual_norm(i["h"].t(), w_pre=i["w_pre"])
    with pytest.raises(ValueError):
        s3d8.residual_norm(i["h"], w_pre=i["w_pre"], h_out=i["h"].clone())
    for bad in (dict(w_post=i["w_post"], w_pre=i["w_pre"]), dict(), dict(gate=i["h"][0, :1], w_pre=i["w_pre"])):
        with pytest.raises(s3d8.S3D8Error) as e:
            s3d8.residual_norm(i["h"], **bad)
        assert e.value.status == -1
    with pytest.raises(s3d8.S3D8Error) as e:       # a gate of another length
        s3d8.residual_norm(i["h"], i["y"], gate=i["w_pre"][:32].clone(), w_pre=i["w_pre"])
    assert e.value.status == -1
    odd = torch.zeros((2, 12), dtype=BF, device=dev())
    with pytest.raises(s3d8.S3D8Error) as e:
        s3d8.residual_norm(odd, w_pre=odd[0].clone())
    assert e.value.status == -1
    flat = torch.zeros((129,), dtype=BF, device=dev())[1:].view(2, 64)
    with pytest.raises(s3d8.S3D8Error) as e:
        s3d8.residual_norm(flat, w_pre=i["w_pre"])
    assert e.value.status == -2
    with pytest.raises(s3d8.S3D8Error) as e:
        s3d8.residual_norm_backward(None, i["h"], i["h"], w_pre=i["w_pre"],
                                    workspace=torch.empty((8,), dtype=torch.uint8, device=dev()))
    assert e.value.status == -6
