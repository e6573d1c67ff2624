"""Normed rotary heads against their formulas in 64 bits, as tensors, as gradients and into
the paged cache, and the gradients against differences.

Tolerances.  A bf16 output is off by its rounding, at most 2^-8 of its size, and by fp32
arithmetic in front of it: two roots' and a dozen operations' errors of 2^-22 and 2^-24 of
the summands' sizes, below 2^-18 of them; the summands of an output column are at most the
row's largest value before the rotation (gradient: before the subtraction) a few times
over.  2^-8 |ref| + 2^-16 of the row's largest value covers both.  An fp32 column sum over m
rows is off by at most (m + 40) 2^-24 of the sum of its summands' sizes.
"""
import numpy as np
import pytest
import torch

import s3d8_a8_linear_gb300 as s3d8
from gpu_util import dev, guarded

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


def _angles(rng, length, rotary):
    a = torch.from_numpy(rng.uniform(-4.0, 4.0, (length, rotary // 2)).astype(np.float32)).to(dev())
    return a.cos(), a.sin()


def _rotate(y, cos, sin, pos, interleaved, back=False):
    """R y (or R^T y) of rows [T, H, D] at positions [T], in y's precision."""
    if cos is None:
        return y
    c, s = cos.double()[pos.long().clamp(min=0)][:, None], sin.double()[pos.long().clamp(min=0)][:, None]
    s = -s if back else s
    r = 2 * c.shape[-1]
    out = y.clone()
    a, b = (y[..., 0:r:2], y[..., 1:r:2]) if interleaved else (y[..., :r // 2], y[..., r // 2:r])
    lo, hi = a * c - b * s, b * c + a * s
    if interleaved:
        out[..., 0:r:2], out[..., 1:r:2] = lo, hi
    else:
        out[..., :r // 2], out[..., r // 2:r] = lo, hi
    return out


def _forward(x, w, cos, sin, pos, interleaved):
    x = x.double()
    y = x if w is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.double()
    z = _rotate(y, cos, sin, pos, interleaved)
    return torch.where((pos >= 0)[:, None, None], z, 0.0), y.abs().amax(-1, keepdim=True)


def _backward(dz, x, w, cos, sin, pos, interleaved):
    """dx, the size of its summands, dw and the sum of its summands' sizes."""
    x = x.double()
    dy = torch.where((pos >= 0)[:, None, None], _rotate(dz.double(), cos, sin, pos, interleaved, back=True), 0.0)
    if w is None:
        return dy, dz.double().abs().amax(-1, keepdim=True), None, None
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    a = dy * w.double()
    dx = r * a - x * r ** 3 * (a * x).mean(-1, keepdim=True)
    size = (r * a.abs()).amax(-1, keepdim=True) + (x.abs() * r ** 3 * (a * x).abs().mean(-1, keepdim=True)).amax(-1, keepdim=True)
    return dx, size, (dy * x * r).sum((0, 1)), (dy * x * r).abs().sum((0, 1))


def _close(got, ref, size):
    excess = (got.double() - ref).abs() - (2.0 ** -8 * ref.abs() + 2.0 ** -16 * size)
    assert (excess <= 0).all(), f"off by {float(excess.max())} beyond the tolerance"


def _close_sum(got, ref, size, rows):
    excess = (got.double() - ref).abs() - (rows + 40) * 2.0 ** -24 * size
    assert (excess <= 0).all(), f"off by {float(excess.max())} beyond the tolerance"


# tokens, query heads, key heads, dim, rotary, interleaved
SIZES = [(1, 1, 0, 16, 0, False), (1, 32, 8, 128, 128, False), (2, 4, 4, 64, 64, True), (3, 3, 1, 80, 80, False),
         (5, 7, 2, 80, 40, False), (7, 5, 1, 256, 256, False), (9, 4, 4, 256, 64, True), (11, 1, 2, 16, 8, False),
         (13, 2, 3, 48, 6, True), (61, 32, 8, 128, 64, False), (300, 8, 0, 128, 0, False), (700, 12, 4, 96, 96, False),
         (1501, 32, 8, 128, 128, False), (5000, 1, 1, 32, 32, True), (40, 100, 50, 112, 12, False)]


def _case(T, Hq, Hk, D, rotary, seed=0, fused=True):
    rng = np.random.default_rng(seed * 1000 + T * 7 + D)
    x = _rand(rng, T, Hq + Hk + 1, D, scale=1.5)       # the heads of one projection, one of them not ours
    q, k = x[:, :Hq], x[:, Hq:Hq + Hk]
    if not fused:
        q, k = q.contiguous(), k.contiguous()
    cos, sin = _angles(rng, T + 5, rotary) if rotary else (None, None)
    pos = torch.from_numpy(rng.permutation(T + 5)[:T].astype(np.int32)).to(dev())
    return rng, q, (k if Hk else None), _rand(rng, D, scale=0.2, mean=1.0), (_rand(rng, D, scale=0.2, mean=1.0) if Hk else None), cos, sin, pos


@pytest.mark.parametrize("T,Hq,Hk,D,rotary,inter", SIZES)
def test_forward(T, Hq, Hk, D, rotary, inter):
    _, q, k, wq, wk, cos, sin, pos = _case(T, Hq, Hk, D, rotary)
    if T > 4:
        pos[1] = -1
    qo, check_q = guarded((T, Hq, D), BF, 3.0)
    ko, check_k = guarded((T, max(Hk, 1), D), BF, 3.0)
    gq, gk = s3d8.norm_rope(q, k, wq, wk, cos, sin, pos, EPS, inter, q_out=qo, k_out=ko if Hk else None)
    torch.cuda.synchronize()
    check_q(), check_k()
    _close(gq, *_forward(q, wq, cos, sin, pos, inter))
    if Hk:
        _close(gk, *_forward(k, wk, cos, sin, pos, inter))
    else:
        assert gk is None


@pytest.mark.parametrize("T,Hq,Hk,D,rotary,inter", SIZES)
def test_backward(T, Hq, Hk, D, rotary, inter):
    rng, q, k, wq, wk, cos, sin, pos = _case(T, Hq, Hk, D, rotary, seed=1)
    if T > 4:
        pos[2] = -7
    dz = _rand(rng, T, Hq + Hk, D)
    dq, dk = dz[:, :Hq], (dz[:, Hq:] if Hk else None)
    g = s3d8.norm_rope_backward(dq, dk, q, k, wq, wk, cos, sin, pos, EPS, inter)
    again = s3d8.norm_rope_backward(dq, dk, q, k, wq, wk, cos, sin, pos, EPS, inter)
    assert set(g) == ({"dq", "dq_norm", "dk", "dk_norm"} if Hk else {"dq", "dq_norm"})
    for n in g:
        assert torch.equal(g[n], again[n]), n
    for dz_, x, w, dx, dw in ((dq, q, wq, "dq", "dq_norm"), (dk, k, wk, "dk", "dk_norm"))[:2 if Hk else 1]:
        ref, size, dw_ref, dw_size = _backward(dz_, x, w, cos, sin, pos, inter)
        _close(g[dx], ref, size)
        _close_sum(g[dw], dw_ref, dw_size, T * x.shape[1])


def test_parts_left_out():
    T, Hq, Hk, D = 37, 6, 2, 64
    rng, q, k, wq, wk, cos, sin, pos = _case(T, Hq, Hk, D, 64, seed=2)
    at = torch.arange(T, device=dev())
    for w1, w2, c, s, p in ((None, wk, cos, sin, pos), (wq, None, cos, sin, None), (None, None, cos, sin, pos),
                            (wq, wk, None, None, pos), (wq, wk, None, None, None)):
        gq, gk = s3d8.norm_rope(q, k, w1, w2, c, s, p)
        where = at if p is None else p
        _close(gq, *_forward(q, w1, c, s, where, False))
        _close(gk, *_forward(k, w2, c, s, where, False))
        dz = _rand(rng, T, Hq + Hk, D)
        g = s3d8.norm_rope_backward(dz[:, :Hq], dz[:, Hq:], q, k, w1, w2, c, s, p)
        assert ("dq_norm" in g) == (w1 is not None) and ("dk_norm" in g) == (w2 is not None)
        _close(g["dq"], *_backward(dz[:, :Hq], q, w1, c, s, where, False)[:2])
        _close(g["dk"], *_backward(dz[:, Hq:], k, w2, c, s, where, False)[:2])
    empty = q[:0]
    gq, gk = s3d8.norm_rope(empty, None, wq, None, cos, sin, pos[:0])
    assert gq.shape == (0, Hq, D) and gk is None
    g = s3d8.norm_rope_backward(empty, None, empty, None, wq, None, cos, sin, pos[:0])
    assert torch.equal(g["dq_norm"], torch.zeros(D, device=dev()))


def test_positions_out_of_range_are_recorded():
    _, q, k, wq, wk, cos, sin, pos = _case(6, 4, 2, 64, 64, seed=3)
    pos[3] = cos.shape[0]
    gq, gk = s3d8.norm_rope(q, k, wq, wk, cos, sin, pos)
    assert s3d8.device_status() == -7
    assert not gq[3].any() and not gk[3].any() and gq[2].any()
    g = s3d8.norm_rope_backward(q, k, q, k, wq, wk, cos, sin, pos)
    assert s3d8.device_status() == -7
    assert not g["dq"][3].any() and not g["dk"][3].any() and g["dq"][4].any()


def test_padding_holds_anything():
    """Rows of padding tokens are never used, not with eps = 0 either."""
    _, q, k, wq, wk, cos, sin, pos = _case(20, 4, 2, 64, 32, seed=4)
    pos[5], pos[11] = -1, -3
    q, k = q.clone(), k.clone()
    clean = [s3d8.norm_rope(q, k, wq, wk, cos, sin, pos, 0.0), s3d8.norm_rope_backward(q, k, q, k, wq, wk, cos, sin, pos, 0.0)]
    for x in (q, k):
        x[5], x[11] = float("nan"), float("inf")
    got = [s3d8.norm_rope(q, k, wq, wk, cos, sin, pos, 0.0), s3d8.norm_rope_backward(q, k, q, k, wq, wk, cos, sin, pos, 0.0)]
    assert all(torch.equal(a, b) for a, b in zip(clean[0], got[0]))
    assert all(torch.equal(clean[1][n], got[1][n]) for n in got[1])


@pytest.mark.parametrize("inter,rotary", [(False, 64), (True, 32), (False, 24)])
def test_gradients_are_those_of_differences(inter, rotary):
    """The formulas above in 64 bits against central differences of the forward one: with
    steps of 2^-13, the second differences leave some 2^-24 of the third derivative."""
    T, H, D = 2, 2, 64
    rng, q, _, wq, _, cos, sin, pos = _case(T, H, 0, D, rotary, seed=5)
    dz = _rand(rng, T, H, D)
    x0, w0, step = q.double(), wq.double(), 2.0 ** -13

    def loss(x, w):
        return float((_forward(x, w, cos, sin, pos, inter)[0] * dz.double()).sum())

    dx, _, dw, _ = _backward(dz, q, wq, cos, sin, pos, inter)
    for i in rng.choice(T * H * D, 40, replace=False):
        e = torch.zeros(T * H * D, dtype=torch.float64, device=dev())
        e[i] = step
        e = e.view(T, H, D)
        assert abs((loss(x0 + e, w0) - loss(x0 - e, w0)) / (2 * step) - float(dx.flatten()[i])) < 1e-5
    for i in rng.choice(D, 20, replace=False):
        e = torch.zeros(D, dtype=torch.float64, device=dev())
        e[i] = step
        assert abs((loss(x0, w0 + e) - loss(x0, w0 - e)) / (2 * step) - float(dw[i])) < 1e-5
    g = s3d8.norm_rope_backward(dz, None, q, None, wq, None, cos, sin, pos, EPS, inter)
    _close(g["dq"], *_backward(dz, q, wq, cos, sin, pos, inter)[:2])


def test_autograd():
    T, Hq, Hk, D = 50, 8, 2, 128
    rng, q, k, wq, wk, cos, sin, pos = _case(T, Hq, Hk, D, 128, seed=6)
    leaves = [t.clone().requires_grad_() for t in (q, k, wq, wk)]
    zq, zk = s3d8.NormRope.apply(*leaves, cos, sin, pos, EPS, False)
    # a gradient that is expanded, and one transposed
    (zq.float().sum() + (zk.transpose(0, 1).float() * 2).sum()).backward()
    one = torch.ones((T, Hq, D), dtype=BF, device=dev())
    want = s3d8.norm_rope_backward(one, 2 * one[:, :Hk].contiguous(), *leaves[:4], cos, sin, pos, EPS, False)
    for leaf, n in zip(leaves, ("dq", "dk", "dq_norm", "dk_norm")):
        assert torch.equal(leaf.grad, want[n].to(BF)), n
    only = q.clone().requires_grad_()
    z, none = s3d8.NormRope.apply(only, None, wq)
    assert none is None
    z.backward(torch.ones_like(z))
    assert torch.equal(only.grad, s3d8.norm_rope_backward(torch.ones_like(z), None, only, None, wq)["dq"])
    with pytest.raises(RuntimeError):
        y, _ = s3d8.NormRope.apply(only, None, wq)
        (first,) = torch.autograd.grad(y.float().square().sum(), only, create_graph=True)
        torch.autograd.grad(first.float().sum(), only)


# into the cache: tokens, query heads, key heads, dim, rotary, interleaved, int8
APPEND = [(1, 4, 1, 64, 64, False, False), (61, 32, 8, 128, 128, False, False), (33, 8, 2, 80, 40, False, False),
          (1700, 32, 8, 128, 128, False, False), (1700, 8, 8, 128, 64, True, False), (900, 6, 2, 256, 256, False, False),
          (61, 32, 8, 128, 128, False, True), (1700, 32, 8, 128, 128, True, True), (700, 4, 4, 80, 12, False, True)]


@pytest.mark.parametrize("T,Hq,Hk,D,rotary,inter,int8", APPEND)
def test_append(T, Hq, Hk, D, rotary, inter, int8):
    rng = np.random.default_rng(T + D)
    x = _rand(rng, T, Hq + 2 * Hk, D, scale=1.5)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]
    wq, wk = _rand(rng, D, scale=0.2, mean=1.0), _rand(rng, D, scale=0.2, mean=1.0)
    page, rows = 16, 3
    each = -(-T // rows)
    width = -(-each // page)
    cos, sin = _angles(rng, each, rotary)
    i = torch.arange(T, device=dev())
    pos, row = (i % each).int(), (i // each).int()
    if T > 4:
        pos[3] = -1
    table = torch.from_numpy(rng.permutation(rows * width).astype(np.int32)).to(dev()).view(rows, width)
    cache = s3d8.KVCache.empty(rows * width, page, Hk, D, torch.int8 if int8 else BF)
    for t in (cache.k, cache.v, *((cache.k_scale, cache.v_scale) if int8 else ())):
        t.zero_()
    got = s3d8.rope_append(q, k, v, cos, sin, pos, cache, table, rows=row, interleaved=inter, q_norm=wq, k_norm=wk, eps=EPS)
    live = pos >= 0
    _close(got, *_forward(q, wq, cos, sin, pos, inter))
    ref, size = _forward(k, wk, cos, sin, pos, inter)
    at = pos.long()[live]
    where = (table[row.long()[live], at // page].long(), at % page)
    if int8:
        # a code is off by half a step of its row, and by one more where fp32 arithmetic in
        # front of it (2^-18 of the largest value) crosses a border
        gk = cache.k[where].double() * cache.k_scale[where].double()[..., None]
        step = ref[live].abs().amax(-1, keepdim=True) / 127
        assert ((gk - ref[live]).abs() <= step * (0.5 + 127 * 2.0 ** -16) + 2.0 ** -16 * size[live]).all()
        plain = s3d8.KVCache.empty(rows * width, page, Hk, D, torch.int8)
        s3d8.rope_append(q, k, v, cos, sin, pos, plain, table, rows=row, interleaved=inter)
        assert torch.equal(cache.v[where], plain.v[where]) and torch.equal(cache.v_scale[where], plain.v_scale[where])
    else:
        _close(cache.k[where], ref[live], size[live])
        assert torch.equal(cache.v[where], v[live])
    # one of the norms alone
    only = s3d8.rope_append(q, k, v, cos, sin, pos, cache, table, rows=row, interleaved=inter, q_norm=wq, eps=EPS)
    assert torch.equal(only, got)
    plain_q = s3d8.rope_append(q, k, v, cos, sin, pos, cache, table, rows=row, interleaved=inter)
    only = s3d8.rope_append(q, k, v, cos, sin, pos, cache, table, rows=row, interleaved=inter, k_norm=wk, eps=EPS)
    assert torch.equal(only, plain_q)


def test_append_padding_with_no_eps():
    rng = np.random.default_rng(9)
    x = _rand(rng, 400, 12, 128)
    cos, sin = _angles(rng, 400, 128)
    pos = torch.arange(400, device=dev()).int()
    pos[::7] = -1
    cache = s3d8.KVCache.empty(25, 16, 2, 128)
    table = torch.arange(25, device=dev()).int().view(1, 25)
    w = _rand(rng, 128, mean=1.0, scale=0.1)
    for n in (5, 400):
        got = s3d8.rope_append(x[:n, :8], x[:n, 8:10], x[:n, 10:], cos, sin, pos[:n], cache, table,
                               rows=torch.zeros(n, dtype=torch.int32, device=dev()), q_norm=w, k_norm=w, eps=0.0)
        assert not got[::7].any() and torch.isfinite(got).all()
