"""The next token at the ends of fp32's range (against the definition of test_gpu_sample)."""
import numpy as np
import pytest
import torch

import s3d8_a8_linear_gb300 as s3d8
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


@pytest.mark.parametrize("V,rows", [(65528, 300), (131056, 300), (262112, 300), (524224, 300), (524224, 3)])
@pytest.mark.parametrize("top,temp", [(17.0, 1.0), (9.0, 0.5), (33.0, 2.0)])
def test_a_heavy_tail_behind_what_is_counted(V, rows, top, temp):
    """A bulk of logits just below exp(-16) of the largest, and enough of exp(-16) that none of the
    bulk is counted.  Each sum of weights is right to 2^-45 of the largest weight for each of its
    tokens, and to 2^-18 of the bulk's weight: so far from its place may a border be."""
    ctas = {65528: 1, 131056: 2, 262112: 4, 524224: 8}[V]
    x = torch.full((V,), 0.98, dtype=BF, device=dev())
    part = -(-(V // ctas) // 8) * 8
    groups = torch.arange(0, 8192, 8 * 4 * ctas, device=dev())          # the tokens that 4 CTAs' worth of lanes read first
    x[(torch.arange(ctas, device=dev())[:, None] * part + groups).flatten()] = 1.0
    x[4321] = top
    y = x.double().cpu().numpy()
    order = np.argsort(-y, kind="stable")
    rank_of = np.empty(V, np.int64)
    rank_of[order] = np.arange(V)
    w = np.exp((y[order] - top) / temp)
    mass = np.cumsum(w)
    head = int((y >= 1.0).sum())
    assert head == 257
    held, tail = mass[-1], mass[-1] - mass[head - 1]
    bound = V * 2.0 ** -45 + 2.0 ** -18 * tail
    rng = np.random.default_rng(V)
    # in front of and behind every third border of the head, and anywhere
    near = np.concatenate([mass[:head:3] / held * (1 + s) for s in (-2.0 ** -24, 2.0 ** -24, -2.0 ** -21)])
    u = np.concatenate((near, rng.random(rows)))[:rows] if rows > 3 else np.array([mass[0] / held, 1 - 2.0 ** -20, 0.97])
    u32 = torch.from_numpy(np.minimum(u, 1 - 2.0 ** -24).astype(np.float32))
    lp = torch.empty(rows, device=dev())
    logits = x.expand(rows, V)
    got = rank_of[s3d8.sample(logits, u32.to(dev()), torch.full((rows,), temp, device=dev()), logprob=lp).cpu().numpy()]
    place = u32.double().numpy() * held
    assert (mass[got] - w[got] <= place + bound).all() and (mass[got] > place - bound).all()
    want = np.log(w[got] / held)
    assert (np.abs(lp.double().cpu().numpy() - want) <= bound / held + 2.0 ** -23 * np.abs(want) + 2.0 ** -25).all()
    # the last token that top-p keeps
    got = rank_of[s3d8.sample(logits, torch.ones(rows, device=dev()), torch.full((rows,), temp, device=dev()), top_p=u32.to(dev())).cpu().numpy()]
    assert (mass[got] >= place - bound).all() and (mass[got] - w[got] < place + bound).all()
