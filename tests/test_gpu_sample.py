"""The next token against the definition in 64 bits, on the CPU.

Tokens are whole numbers and have to be equal.  Weights are whole numbers of 2^-45, so a
border between two tokens lies within about 2^-45 of its place; a given u (a multiple of
2^-24) falls between a border and its place once in some 2^20 rows of thousands of tokens
here.  logprob is fp32 from 64-bit arithmetic on sums that are right to 2^-28: within 2^-24
of its size and 2^-26.
"""
import numpy as np
import pytest
import torch

import s3d8_a8_linear_gb300 as s3d8
from gpu_util import dev, guarded

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    s3d8.load(build_if_missing=True)
    torch.cuda.set_device(0)
    yield
    assert s3d8.device_status() == 0


def _one(x, u, temp=1.0, k=0, p=1.0, m=0.0):
    """Token and logprob of one row of float64 logits."""
    x = np.where(np.isnan(x), -np.inf, x)
    if not (x > -np.inf).any():
        return -1, -np.inf
    top = x.max()
    if not temp > 0:
        return int(np.flatnonzero(x == top)[0]), 0.0
    order = np.argsort(-x, kind="stable")
    order = order[x[order] > -np.inf]
    with np.errstate(over="ignore", invalid="ignore"):
        gap = np.where(x[order] == top, 0.0, (x[order] - top) / temp)
    w = np.exp(gap)
    n = min(k, len(w)) if k > 0 else len(w)
    mass = np.cumsum(w)
    if p < 1:
        n = min(n, int((mass[:n] < p * mass[n - 1]).sum()) + 1)
    n = min(n, max(1, int((w >= m).sum())))
    r = min(int((mass[:n] <= u * mass[n - 1]).sum()), n - 1)
    return int(order[r]), gap[r] - np.log(mass[n - 1])


def _check(logits, u, temp=None, k=None, p=None, m=None):
    B = logits.shape[0]

    def t(a, dtype):
        return None if a is None else torch.as_tensor(np.broadcast_to(np.asarray(a), (B,)).copy(), dtype=dtype, device=dev())

    temp, p, m = (t(a, torch.float32) for a in (temp, p, m))
    k, u = t(k, torch.int32), t(u, torch.float32)
    out, check = guarded((B,), torch.int32, 77)
    lp, check_lp = guarded((B,), torch.float32, 7.0)
    got = s3d8.sample(logits, u, temp, k, p, m, tokens=out, logprob=lp)
    torch.cuda.synchronize()
    check(), check_lp()
    assert torch.equal(got, s3d8.sample(logits, u, temp, k, p, m))
    x = logits.float().cpu().numpy().astype(np.float64)

    def v(a, i, none):
        return none if a is None else a[i].item()

    for i in range(B):
        token, logprob = _one(x[i], v(u, i, 0), v(temp, i, 1.0), v(k, i, 0), v(p, i, 1.0), v(m, i, 0.0))
        assert int(got[i]) == token, (i, int(got[i]), token)
        if np.isfinite(logprob):
            assert abs(float(lp[i]) - logprob) <= 2.0 ** -23 * abs(logprob) + 2.0 ** -25, i
        else:
            assert float(lp[i]) == logprob, i
    return got


def _logits(rng, B, V, spread=3.0):
    return torch.from_numpy((spread * rng.standard_normal((B, V))).astype(np.float32)).to(BF).to(dev())


VOCABS = [1, 2, 7, 8, 9, 255, 1000, 8191, 8192, 8193, 20001, 65528, 65535, 128256]


@pytest.mark.parametrize("V", VOCABS)
@pytest.mark.parametrize("limits", ["none", "k", "p", "m", "all"])
def test_against_the_definition(V, limits):
    rng = np.random.default_rng(V)
    B = 13
    i = np.arange(B)
    _check(_logits(rng, B, V), rng.random(B), 0.5 + 0.1 * i,
           k=1 + (i * 53) % max(1, V) if limits in ("k", "all") else None,
           p=rng.random(B) if limits in ("p", "all") else None,
           m=10.0 ** -rng.uniform(0, 6, B) if limits in ("m", "all") else None)


@pytest.mark.parametrize("B,V", [(200, 4000), (90, 65528), (90, 65529), (45, 128256), (25, 128256), (3, 131056), (2, 131057),
                                 (80, 131056), (2, 262144), (41, 262112), (1, 524224), (500, 9000)])
def test_rows_and_clusters(B, V):
    """Every number of CTAs that a row may get."""
    rng = np.random.default_rng(B)
    _check(_logits(rng, B, V, 2.0), rng.random(B), np.where(np.arange(B) % 9 == 8, 0.0, 0.8),
           k=np.where(np.arange(B) % 3 == 0, 40, 0), p=np.where(np.arange(B) % 2 == 0, 0.9, 1.0))


def test_equal_logits_divide_evenly():
    """Equal weights are exact: u = j / V is the border in front of token j."""
    for V in (8, 64, 16384):
        x = torch.full((1, V), 1.5, dtype=BF, device=dev())
        for j in (0, 1, 3, V // 2, V - 1):
            assert int(_check(x, j / V)) == j
            assert int(_check(x, (j + 1) / V - 2.0 ** -24)) == j
        assert int(_check(x, 1.0 - 2.0 ** -24, p=0.5)) == V // 2 - 1     # half of the weight: half of the tokens
        assert int(_check(x, 1.0 - 2.0 ** -24, k=3)) == 2
        assert int(_check(x, 1.0 - 2.0 ** -24, k=4, p=0.5)) == 1
        assert int(_check(x, 0.9, m=1.0)) == int(0.9 * V) and int(_check(x, 0.9, m=1.5)) == 0
    x = torch.full((1, 524224), -2.0, dtype=BF, device=dev())       # the largest sum of weights
    assert int(_check(x, 0.999)) == int(np.float32(0.999).astype(np.float64) * 524224)


def test_edges_of_the_limits():
    rng = np.random.default_rng(5)
    x = _logits(rng, 1, 3000)
    first = int(x[0].float().argmax())
    for p in (0.0, -1.0, 1e-30):
        assert int(_check(x, 0.99, p=p)) == first
    for k in (1, 0, -5, 3000, 10 ** 9):
        _check(x, 0.7, k=k)
    for u in (0.0, 1.0, 2.0, 1.0 - 2.0 ** -24, 2.0 ** -24, 1e-30):
        _check(x, u)
        _check(x, u, k=50, p=0.8, m=0.01)
    for temp in (0.0, -1.0, float("nan"), 1e-30, 1e-45, 1e-3, 100.0, 1e30, float("inf")):
        _check(x, 0.3, temp)
    assert int(_check(x, 0.5, 1e-20)) == first


def test_values_that_are_not_numbers():
    inf, nan = float("inf"), float("nan")
    low = torch.finfo(BF).min
    rows = [[-inf] * 9, [nan] * 9, [nan, -inf] * 4 + [1.0], [inf, 1, inf, 0, inf, 2, 3, 4, 5], [low] * 9,
            [low, 3.0, low, 2.0, low, low, 1.0, low, low], [0.0, -0.0, 0.0, -0.0, -1.0, -0.0, 0.0, 0.0, -0.0],
            [-0.0, 0.0, nan, -inf, inf, low, 1.0, 2.0, 3.0], [1e-40, -1e-40, 1e-39, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0]]
    x = torch.tensor(rows, dtype=torch.float32).to(BF).to(dev())
    for u in (0.0, 0.3, 0.77, 1 - 2.0 ** -24):
        for temp in (1.0, 0.0, 0.5):
            got = _check(x, u, temp)
            assert int(got[0]) == -1 and int(got[1]) == -1 and int(got[2]) == 8
            _check(x, u, temp, k=3)
            _check(x, u, temp, p=0.6)
            _check(x, u, temp, m=0.5)


def test_banned_words_are_never_drawn():
    rng = np.random.default_rng(6)
    x = _logits(rng, 40, 128256)
    ban = torch.rand(x.shape, device=dev()) < 0.5
    x = x.masked_fill(ban, -float("inf"))
    got = _check(x, rng.random(40), 1.3, p=0.99)
    assert not ban.gather(1, got.long()[:, None]).any()


def test_rows_apart_and_unaligned():
    rng = np.random.default_rng(7)
    wide = _logits(rng, 12, 10007)
    for x in (wide[:, :9999], wide[:, 1:10000], wide[::3, 3:9003], wide[:1, 5:6], wide.expand(12, 10007)[2:3]):
        _check(x, rng.random(x.shape[0]), 0.9, k=200)
    same = wide[:1].expand(5, 10007)
    _check(same, rng.random(5), 1.1)


def test_shares_are_those_of_the_weights():
    """Evenly spread u draw each token by its share: the counts over 2^14 of them are within
    one of 2^14 p."""
    n = 1 << 14
    x = torch.tensor([2.0, -1.0, 0.5, 1.0, -3.0, 0.0, 1.5, 0.25], dtype=BF, device=dev())
    u = (torch.arange(n, device=dev()).float() + 0.5) / n
    got = s3d8.sample(x.expand(n, 8), u)
    share = torch.softmax(x.double(), 0) * n
    assert ((torch.bincount(got.long(), minlength=8) - share).abs() <= 1).all()


def test_no_rows_and_captured():
    assert s3d8.sample(torch.empty((0, 100), dtype=BF, device=dev()), torch.empty(0, device=dev())).shape == (0,)
    rng = np.random.default_rng(8)
    x, u = _logits(rng, 30, 50000), torch.rand(30, device=dev())
    out = torch.empty(30, dtype=torch.int32, device=dev())
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        s3d8.sample(x, u, tokens=out)
    stream.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s3d8.sample(x, u, tokens=out)
        s3d8.sample(x, u, tokens=out)
    for _ in range(3):
        u.copy_(torch.rand(30, device=dev()))
        x.copy_(_logits(rng, 30, 50000))
        g.replay()
        torch.cuda.synchronize()
        _check(x, u.cpu().numpy())
        assert torch.equal(out, s3d8.sample(x, u))
