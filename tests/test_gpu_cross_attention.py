"""Cross attention and its gradients against their formulas in 64 bits, and the gradients
against differences.

Tolerances.  Scores are fp32 sums of dim exact products: with the exponential's 2^-22 and
the arithmetic around it, a weight p_j is right to 2^-12 of itself while scale * |q| . |k|
stays below 30, as here ((dim + 4) 2^-24 30 < 2^-12.9).  On its way into the product with
the values it is rounded to bf16, 2^-8 of it.  So

  |out - ref| <= (2^-8 + 2^-12) sum_j p_j |v_j| + 2^-8 |ref|   (the last for its own rounding).

dv likewise with |dout| for |v|.  ds_j = p_j (dout . v_j - delta) is right to 2^-12 of
A_j = p_j (sum |dout| |v_j| + sum |dout| |out|), or of p_j (sum |dout| |v_j| + sum_i p_i sum
|dout| |v_i|) where delta is summed from its parts, and is rounded to bf16 for the products with k
and q:  |dq - ref| <= scale sum_j (2^-8 |ds_j| + 2^-11 A_j) |k_j| + 2^-8 |ref|, dk likewise.
The fp32 sums over up to n tokens or states add n 2^-24 of the summands' sizes, below 2^-11
of them here.  lse: 2^-13 (its scores' error) and 2^-22 of its size.
"""
import pytest
import torch

import s3d8_a8_linear_gb300 as s3d8
from gpu_util import guarded

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


def _rand(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda").to(BF)


def _reference(q, k, v, spans, scale, dout=None, out=None):
    """The formulas in 64 bits, a query head at a time, and the tolerances that go with them."""
    T, Hq, D = q.shape
    S, heads = k.shape[:2]
    group = Hq // heads
    f64 = dict(dtype=torch.float64, device=q.device)
    r = {n: torch.zeros((T, Hq, D), **f64) for n in ("out", "out_tol", "dq", "dq_tol")}
    r.update({n: torch.zeros((S, heads, D), **f64) for n in ("dk", "dk_tol", "dv", "dv_tol")})
    r["lse"] = torch.full((T, Hq), -float("inf"), **f64)
    j = torch.arange(S, device=q.device)
    if spans is None:
        seen = torch.ones((T, S), dtype=torch.bool, device=q.device)
    else:
        seen = (j >= spans[:, :1]) & (j < spans[:, 1:])
    for h in range(Hq):
        g = h // group
        Q, K, V = q[:, h].double(), k[:, g].double(), v[:, g].double()
        # what nobody sees has no part in anything
        K, V = (torch.where(seen.any(0)[:, None], x, 0.0) for x in (K, V))
        Q = torch.where(seen.any(1)[:, None], Q, 0.0)
        s = (scale * Q @ K.T).masked_fill(~seen, -float("inf"))
        r["lse"][:, h] = torch.logsumexp(s, -1)
        p = torch.where(seen, torch.exp(s - r["lse"][:, h].clamp(min=-1e300)[:, None]), 0.0)
        r["out"][:, h] = p @ V
        r["out_tol"][:, h] = (2.0 ** -8 + 2.0 ** -12) * (p @ V.abs()) + 2.0 ** -8 * r["out"][:, h].abs() + 1e-30
        if dout is None:
            continue
        dO, O = dout[:, h].double(), out[:, h].double()
        dO = torch.where(seen.any(1)[:, None], dO, 0.0)
        # a token of at most 128 states: delta is summed from p_j (dout . v_j), each right to 2^-12
        # of p_j sum |dout| |v_j|; else it is that of the given output
        few = (seen.sum(1) <= 128)[:, None]
        size = dO.abs() @ V.abs().T
        delta = torch.where(few, (p * (dO @ V.T)).sum(-1, keepdim=True), (dO * O).sum(-1, keepdim=True))
        ds = p * (dO @ V.T - delta)
        A = p * (size + torch.where(few, (p * size).sum(-1, keepdim=True), (dO * O).abs().sum(-1, keepdim=True)))
        e = abs(scale) * (2.0 ** -8 * ds.abs() + 2.0 ** -11 * A)
        r["dq"][:, h] = scale * ds @ K
        r["dq_tol"][:, h] = e @ K.abs()
        r["dk"][:, g] += scale * ds.T @ Q
        r["dk_tol"][:, g] += e.T @ Q.abs()
        r["dv"][:, g] += p.T @ dO
        r["dv_tol"][:, g] += (2.0 ** -8 + 2.0 ** -11) * (p.T @ dO.abs())
    for n in ("dq", "dk", "dv"):
        r[n + "_tol"] += 2.0 ** -8 * r[n].abs() + 1e-30
    return r


def _within(got, ref, tol, what):
    assert torch.isfinite(got).all(), what
    excess = (got.double() - ref).abs() - tol
    assert (excess <= 0).all(), f"{what}: off by {float(excess.max())} beyond the tolerance"


def _within_lse(got, ref):
    assert torch.equal(torch.isfinite(got), torch.isfinite(ref)) and not torch.isnan(got).any()
    some = torch.isfinite(ref)
    assert ((got.double() - ref)[some].abs() <= 2.0 ** -13 + 2.0 ** -22 * ref[some].abs()).all()
    assert (got[~some] == -float("inf")).all()


def _check(q, k, v, spans=None, scale=None, back=True):
    """Forward and gradients of one call; the outputs."""
    T, Hq, D = q.shape
    S, heads = k.shape[:2]
    gen = torch.Generator(device="cuda").manual_seed(T * 7 + S)
    out, c1 = guarded((T, Hq, D), BF, 3.0)
    lse, c2 = guarded((T, Hq), torch.float32, 3.0)
    space = s3d8.cross_attention_workspace(T, S, Hq, heads, D).fill_(0xFF)       # NaN, whatever is read of it first
    s3d8.cross_attention(q, k, v, spans, scale, out=out, lse=lse, workspace=space)
    torch.cuda.synchronize()
    c1(), c2()
    alone = s3d8.cross_attention(q, k, v, spans, scale, workspace=space)
    assert torch.equal(out, alone), "two calls differ, or lse changes the output"
    dout = _rand(gen, T, Hq, D) if back else None
    r = _reference(q, k, v, spans, D ** -0.5 if scale is None else scale, dout, out)
    _within(out, r["out"], r["out_tol"], "out")
    _within_lse(lse, r["lse"])
    got = {"out": out, "lse": lse}
    if back:
        space = s3d8.cross_attention_backward_workspace(T, S, Hq, heads, D).fill_(0xFF)
        g = s3d8.cross_attention_backward(dout, q, k, v, out, lse, spans, scale, workspace=space)
        again = s3d8.cross_attention_backward(dout, q, k, v, out, lse, spans, scale, workspace=space)
        for n in ("dv", "dk", "dq"):
            assert torch.equal(g[n], again[n]), n
            _within(g[n], r[n], r[n + "_tol"], n)
        got.update(g)
    return got


def _random_spans(gen, T, S, kind):
    if kind is None:
        return None
    lo = torch.randint(0, S + 1, (T,), generator=gen, device="cuda")
    hi = torch.randint(0, S + 1, (T,), generator=gen, device="cuda")
    if kind == "any":           # a half of them empty
        return torch.stack((lo, hi), -1).int()
    if kind == "images":        # a few images, each token one of them, in order
        n = min(4, S)
        at = torch.arange(T, device="cuda") * n // T
        return torch.stack((at * (S // n), (at + 1) * (S // n)), -1).int()
    if kind == "one":           # a single state each
        lo = lo.clamp(max=S - 1)
        return torch.stack((lo, lo + 1), -1).int()
    if kind == "none":
        return torch.stack((lo, lo), -1).int()
    raise AssertionError(kind)


# tokens, states, query heads, key/value heads, dim
SIZES = [(1, 1, 1, 1, 8), (1, 1601, 32, 8, 128), (1, 127, 4, 4, 64), (1, 129, 8, 2, 80), (2, 128, 16, 1, 128), (3, 300, 5, 1, 96),
         (7, 1000, 14, 2, 64), (31, 33, 4, 1, 16), (32, 257, 8, 2, 128), (33, 640, 4, 1, 128), (64, 512, 4, 2, 64),
         (65, 400, 6, 2, 40), (127, 129, 1, 1, 128), (128, 128, 2, 2, 128), (129, 385, 3, 1, 72), (200, 77, 128, 1, 64),
         (255, 1601, 8, 2, 128), (257, 900, 2, 1, 80), (513, 514, 4, 4, 128), (1000, 130, 4, 1, 24), (90, 3000, 10, 2, 128)]


@pytest.mark.parametrize("kind", [None, "any", "images", "one"])
@pytest.mark.parametrize("T,S,Hq,heads,dim", SIZES)
def test_sizes(T, S, Hq, heads, dim, kind):
    gen = torch.Generator(device="cuda").manual_seed(T + S)
    q, both = _rand(gen, T, Hq, dim), _rand(gen, S, 2 * heads, dim)
    _check(q, both[:, :heads], both[:, heads:], _random_spans(gen, T, S, kind))


@pytest.mark.parametrize("T,S,dim", [(1, 9, 64), (70, 300, 128), (300, 70, 80)])
def test_tokens_that_see_nothing(T, S, dim):
    gen = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = _rand(gen, T, 4, dim), _rand(gen, S, 2, dim), _rand(gen, S, 2, dim)
    spans = _random_spans(gen, T, S, "none")
    got = _check(q, k, v, spans)
    assert not got["out"].any() and (got["lse"] == -float("inf")).all()
    assert not any(got[n].any() for n in ("dq", "dk", "dv"))
    spans[T // 2] = torch.tensor([2, 5], device="cuda")        # one that does, among them
    got = _check(q, k, v, spans)
    assert got["dk"][2:5].any() and not got["dk"][5:].any() and not got["dv"][:2].any()


def test_no_states_and_no_tokens():
    gen = torch.Generator(device="cuda").manual_seed(2)
    q, k = _rand(gen, 5, 4, 64), _rand(gen, 3, 2, 64)
    lse = torch.empty((5, 4), device="cuda")
    out = s3d8.cross_attention(q, k[:0], k[:0], lse=lse)
    assert not out.any() and (lse == -float("inf")).all()
    g = s3d8.cross_attention_backward(q, q, k[:0], k[:0], out, lse)
    assert not g["dq"].any() and g["dk"].shape == (0, 2, 64)
    out = s3d8.cross_attention(q[:0], k, k)
    assert out.shape == (0, 4, 64)
    g = s3d8.cross_attention_backward(q[:0], q[:0], k, k, out, lse[:0])
    assert not g["dk"].any() and not g["dv"].any() and g["dk"].shape == k.shape


def test_spans_out_of_range_are_cut_and_recorded():
    gen = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = _rand(gen, 40, 4, 64), _rand(gen, 200, 1, 64), _rand(gen, 200, 1, 64)
    spans = torch.tensor([[-5, 60], [100, 900], [-9, 400], [300, 400], [-8, -3]], device="cuda").int().repeat(8, 1)
    lse = torch.empty((40, 4), device="cuda")
    out = s3d8.cross_attention(q, k, v, spans, lse=lse)
    assert s3d8.device_status() == -7
    cut = spans.clamp(0, 200)
    assert torch.equal(out, s3d8.cross_attention(q, k, v, cut))
    g = s3d8.cross_attention_backward(q, q, k, v, out, lse, spans)
    assert s3d8.device_status() == -7
    want = s3d8.cross_attention_backward(q, q, k, v, out, lse, cut)
    assert all(torch.equal(g[n], want[n]) for n in g)
    backwards = torch.tensor([[900, -5]], device="cuda").int().repeat(40, 1)       # empty, wherever it lies
    assert not s3d8.cross_attention(q, k, v, backwards).any() and s3d8.device_status() == 0


@pytest.mark.parametrize("T,group,bad", [(3, 4, float("nan")), (40, 4, float("inf")), (300, 1, float("nan")), (48, 4, -float("inf"))])
def test_states_behind_a_span_hold_anything(T, group, bad):
    """Padding between the images, of NaN or infinities, changes nothing."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    S, dim = 1000, 128
    q, k, v = _rand(gen, T, 2 * group, dim), _rand(gen, S, 2, dim), _rand(gen, S, 2, dim)
    at = torch.arange(T, device="cuda") % 3
    spans = torch.stack((at * 333, at * 333 + 150 + 50 * at), -1).int()
    clean = _check(q, k, v, spans)
    j = torch.arange(S, device="cuda")
    unseen = ~((j >= spans[:, :1]) & (j < spans[:, 1:])).any(0)
    k, v = k.clone(), v.clone()
    k[unseen], v[unseen] = bad, bad
    got = _check(q, k, v, spans)
    assert all(torch.equal(clean[n], got[n]) for n in ("out", "lse", "dq"))
    assert torch.equal(clean["dk"], got["dk"]) and torch.equal(clean["dv"], got["dv"])


@pytest.mark.parametrize("T,S,share", [(12, 120, 10), (48, 2000, 40), (300, 900, 3)])
def test_one_sequence_does_not_reach_another(T, S, share):
    """Infinities and NaN among one sequence's values are that sequence's alone, column by
    column as the sum has them."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    q, k, v = _rand(gen, T, 4, 64), _rand(gen, S, 1, 64), _rand(gen, S, 1, 64)
    first = (torch.arange(T, device="cuda") * (S // T)).int()
    spans = torch.stack((first, first + share), -1).int().clamp(max=S)
    clean = s3d8.cross_attention(q, k, v, spans)
    bad = v.clone()
    j = int(first[T // 2]) + 1
    bad[j, 0, 3], bad[j, 0, 9], bad[j, 0, 11] = float("nan"), float("inf"), -float("inf")
    bad[j + 1, 0, 11] = float("inf")
    got = s3d8.cross_attention(q, k, bad, spans)
    for t in range(T):
        sees = [bool(spans[t, 0] <= i < spans[t, 1]) for i in (j, j + 1)]
        want = clean[t].clone()
        if sees[0]:
            want[:, 3], want[:, 9], want[:, 11] = float("nan"), float("inf"), -float("inf")
        if sees[1]:
            want[:, 11] = float("nan") if sees[0] else float("inf")
        assert torch.equal(torch.nan_to_num(got[t], 1e4, 2e4, -2e4), torch.nan_to_num(want, 1e4, 2e4, -2e4)), t


def test_keys_of_one_sequence_do_not_reach_another():
    gen = torch.Generator(device="cuda").manual_seed(6)
    T, S = 20, 400
    q, k, v = _rand(gen, T, 4, 64), _rand(gen, S, 1, 64), _rand(gen, S, 1, 64)
    first = (torch.arange(T, device="cuda") * 20).int()
    spans = torch.stack((first, first + 20), -1).int()
    clean = s3d8.cross_attention(q, k, v, spans)
    k[205], q[3] = float("nan"), float("inf")
    got = s3d8.cross_attention(q, k, v, spans)
    others = [t for t in range(T) if t not in (3, 10)]
    assert torch.equal(got[others], clean[others]) and torch.isnan(got[10]).all() and torch.isnan(got[3]).all()


@pytest.mark.parametrize("scale", [0.0, 1e-3, 0.5, -0.125])
def test_scales(scale):
    gen = torch.Generator(device="cuda").manual_seed(7)
    q, k, v = _rand(gen, 50, 4, 64) * 0.5, _rand(gen, 300, 2, 64), _rand(gen, 300, 2, 64)
    _check(q, k, v, None, scale)


def test_scores_of_all_sizes():
    """Scores far apart, and a maximum that keeps rising from state to state: the weights
    follow the running maximum.  (Scores of up to 300, of one product each and so exact: the
    rounding of their base-2 exponents, 300 * 1.45 * 2^-24, is within the 2^-12 of the
    tolerances' weights.)"""
    S = 700
    q = torch.zeros((130, 1, 64), dtype=BF, device="cuda")
    q[:, 0, 0] = 8.0
    k, v = torch.zeros((S, 1, 64), dtype=BF, device="cuda"), _rand(torch.Generator(device="cuda").manual_seed(8), S, 1, 64)
    for turn in (1, -1):
        k[:, 0, 0] = torch.linspace(-300, 300, S, device="cuda").to(BF) * turn
        _check(q, k, v)
    k[:, 0, 0] = 0
    k[699, 0, 0] = 300.0
    _check(q, k, v)


def test_strides():
    T, S, D = 70, 333, 64
    gen = torch.Generator(device="cuda").manual_seed(9)
    q, k, v = _rand(gen, T, 8, D), _rand(gen, S, 2, D), _rand(gen, S, 2, D)
    base = _check(q, k, v)
    wide = torch.full((T, 9, 2 * D), 7.0, dtype=BF, device="cuda")
    wide[:, 1:, D:] = q
    turned = k.transpose(0, 1).contiguous().transpose(0, 1)         # head-major
    every = torch.full((2 * S, 2, D), 7.0, dtype=BF, device="cuda")
    every[::2] = v
    got = _check(wide[:, 1:, D:], turned, every[::2])
    assert all(torch.equal(base[n], got[n]) for n in base)
    one = _rand(gen, 1, 1, D).expand(S, 2, D)                       # the same row for every state and head
    _check(q, one, v)
    _check(q, k, one)
    _check(_rand(gen, 1, 1, D).expand(T, 8, D), k, v)


def test_spans_may_be_in_any_order():
    gen = torch.Generator(device="cuda").manual_seed(10)
    T, S = 400, 2000
    q, k, v = _rand(gen, T, 4, 128), _rand(gen, S, 1, 128), _rand(gen, S, 1, 128)
    lo = torch.randint(0, S - 50, (T,), generator=gen, device="cuda")
    spans = torch.stack((lo, lo + 50), -1).int()
    got = _check(q, k, v, spans)
    order = torch.randperm(T, generator=gen, device="cuda")
    turned = s3d8.cross_attention(q[order], k, v, spans[order])
    r = _reference(q, k, v, spans, 128 ** -0.5)
    _within(turned, r["out"][order], r["out_tol"][order], "out")
    assert got["out"].shape == turned.shape


@pytest.mark.parametrize("batch,tokens,states,Hq,heads,dim", [(48, 1, 900, 32, 8, 128), (5, 333, 401, 16, 16, 80),
                                                             (3, 700, 1601, 8, 2, 128), (100, 2, 70, 4, 1, 64)])
def test_batches(batch, tokens, states, Hq, heads, dim):
    """Sequences one behind the other, of unlike numbers of states, some without any."""
    gen = torch.Generator(device="cuda").manual_seed(batch)
    T, S = batch * tokens, batch * states
    q, k, v = _rand(gen, T, Hq, dim), _rand(gen, S, heads, dim), _rand(gen, S, heads, dim)
    real = torch.randint(0, states + 1, (batch,), generator=gen, device="cuda")
    real[0], real[-1] = states, 0
    first = (torch.arange(batch, device="cuda") * states)[:, None].expand(batch, tokens)
    spans = torch.stack((first, first + real[:, None]), -1).view(T, 2).int()
    _check(q, k, v, spans)


def test_gradients_are_those_of_differences():
    """The formulas' gradients against central differences of the formulas' output, in 64
    bits; with steps of 2^-13 the differences are right to some 1e-6."""
    gen = torch.Generator(device="cuda").manual_seed(11)
    T, S, D = 3, 5, 8
    q, k, v = _rand(gen, T, 2, D), _rand(gen, S, 1, D), _rand(gen, S, 1, D)
    spans = torch.tensor([[0, 5], [1, 4], [2, 2]], device="cuda").int()
    dout, scale, step = _rand(gen, T, 2, D), 0.4, 2.0 ** -13
    exact = _reference(q, k, v, spans, scale)["out"]
    r = _reference(q, k, v, spans, scale, dout, exact)

    def loss(**change):
        x = {"q": q.double(), "k": k.double(), "v": v.double(), **change}
        return float((_reference(x["q"], x["k"], x["v"], spans, scale)["out"] * dout.double()).sum())

    for name, x in (("q", q), ("k", k), ("v", v)):
        for i in range(x.numel()):
            e = torch.zeros(x.numel(), dtype=torch.float64, device="cuda")
            e[i] = step
            e = e.view(x.shape)
            diff = (loss(**{name: x.double() + e}) - loss(**{name: x.double() - e})) / (2 * step)
            assert abs(diff - float(r["d" + name].flatten()[i])) < 1e-5, (name, i)
    _check(q, k, v, spans, scale)


def test_autograd():
    gen = torch.Generator(device="cuda").manual_seed(12)
    q, k, v = _rand(gen, 60, 4, 64), _rand(gen, 150, 2, 64), _rand(gen, 150, 2, 64)
    spans = _random_spans(gen, 60, 150, "images")
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    out = s3d8.CrossAttention.apply(*leaves, spans)
    out.float().sum().backward()                # an expanded gradient
    lse = torch.empty((60, 4), device="cuda")
    o = s3d8.cross_attention(q, k, v, spans, lse=lse)
    want = s3d8.cross_attention_backward(torch.ones_like(o), q, k, v, o, lse, spans)
    for leaf, n in zip(leaves, ("dq", "dk", "dv")):
        assert torch.equal(leaf.grad, want[n])
    with pytest.raises(RuntimeError):
        out = s3d8.CrossAttention.apply(*leaves, spans, 0.2)
        (first,) = torch.autograd.grad(out.float().square().sum(), leaves[0], create_graph=True)
        torch.autograd.grad(first.float().sum(), leaves[1])


def test_other_stream_and_captured():
    gen = torch.Generator(device="cuda").manual_seed(13)
    q, k, v = _rand(gen, 300, 8, 128), _rand(gen, 1500, 2, 128), _rand(gen, 1500, 2, 128)
    spans = _random_spans(gen, 300, 1500, "images")
    dout = _rand(gen, 300, 8, 128)
    lse, out = torch.empty((300, 8), device="cuda"), torch.empty_like(q)
    want = s3d8.cross_attention(q, k, v, spans, lse=lse)
    grads = s3d8.cross_attention_backward(dout, q, k, v, want, lse, spans)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    space, back = s3d8.cross_attention_workspace(300, 1500, 8, 2, 128), s3d8.cross_attention_backward_workspace(300, 1500, 8, 2, 128)
    with torch.cuda.stream(side):
        s3d8.cross_attention(q, k, v, spans, out=out, workspace=space)
    side.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s3d8.cross_attention(q, k, v, spans, out=out, lse=lse, workspace=space)
        got = s3d8.cross_attention_backward(dout, q, k, v, out, lse, spans, workspace=back)
    for _ in range(3):
        out.fill_(0)
        lse.fill_(0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and all(torch.equal(got[n], grads[n]) for n in got)


def test_far_states():
    """Offsets past 2^31 elements."""
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB")
    S, dim = (1 << 24) - 5, 128
    both = torch.empty((S, 2, dim), dtype=BF, device="cuda")        # 4.3 billion elements
    gen = torch.Generator(device="cuda").manual_seed(14)
    both[-700:] = _rand(gen, 700, 2, dim)
    both[:300] = _rand(gen, 300, 2, dim)
    q = _rand(gen, 6, 2, dim)
    spans = torch.tensor([[S - 700, S], [S - 300, S - 1], [0, 300]] * 2, device="cuda").int()
    near = torch.cat((both[:300], both[-700:]))
    moved = torch.where(spans >= 1000, spans - (S - 1000), spans)
    out = s3d8.cross_attention(q, both[:, :1], both[:, 1:], spans)
    r = _reference(q, near[:, :1], near[:, 1:], moved, dim ** -0.5)
    _within(out, r["out"], r["out_tol"], "out")


@pytest.mark.parametrize("T,group,kind", [(1, 4, "gaps"), (48, 4, "gaps"), (200, 1, "gaps"), (97, 8, "gaps"), (1000, 4, "gaps"), (700, 128, "gaps"),
                                          (64, 4, "behind"), (513, 2, "behind")])
def test_states_that_nobody_sees(T, group, kind):
    """Sequences of their own states, most of which are padding: whole tiles between the ones
    that are seen hold NaN, and the visits of a query tile jump over them."""
    gen = torch.Generator(device="cuda").manual_seed(T)
    heads, dim, S = 2, 64, 60000
    t = torch.arange(T, device="cuda")
    if kind == "gaps":          # token t's states begin anywhere in its share of them, and are few
        share = S // T
        lo = t * share + torch.randint(0, max(share // 2, 1), (T,), generator=gen, device="cuda")
        hi = torch.minimum(lo + torch.randint(0, 300, (T,), generator=gen, device="cuda"), (t + 1) * share)
    else:                       # far first, near last
        lo = (T - 1 - t) * (S // T)
        hi = lo + 37
    spans = torch.stack((lo, hi), -1).int()
    q, k, v = _rand(gen, T, heads * group, dim), _rand(gen, S, heads, dim), _rand(gen, S, heads, dim)
    seen = torch.zeros(S + 1, dtype=torch.int32, device="cuda")
    seen.index_add_(0, spans[:, 0].long(), torch.ones(T, dtype=torch.int32, device="cuda"))
    seen.index_add_(0, spans[:, 1].long(), -torch.ones(T, dtype=torch.int32, device="cuda"))
    unseen = seen.cumsum(0)[:S] == 0
    k[unseen] = float("nan")
    v[unseen] = float("nan")
    out = torch.full_like(q, 3.0)
    lse = torch.full((T, heads * group), 3.0, device="cuda")
    s3d8.cross_attention(q, k, v, spans, out=out, lse=lse)
    for i in range(0, T, max(1, T // 40)):
        a, b = spans[i].tolist()
        r = _reference(q[i:i + 1], k[a:b], v[a:b], None, dim ** -0.5) if b > a else None
        if r is None:
            assert not out[i].any() and bool((lse[i] == -float("inf")).all())
        else:
            _within(out[i:i + 1], r["out"], r["out_tol"], f"token {i}")
            _within_lse(lse[i:i + 1], r["lse"])


def test_more_tiles_than_a_launch():
    """Gradients with more query tiles and more tiles of states than one launch sums up (128
    of either), ragged at both ends."""
    gen = torch.Generator(device="cuda").manual_seed(9)
    T, S, heads, group, dim = 4237, 16999, 1, 4, 64
    q, k, v = _rand(gen, T, heads * group, dim), _rand(gen, S, heads, dim), _rand(gen, S, heads, dim)
    at = torch.arange(T, device="cuda") * 5 // T
    spans = torch.stack((at * (S // 5), at * (S // 5) + S // 5 - 7 * at), -1).int()
    _check(q, k, v, spans)


@pytest.mark.parametrize("dim", [64, 128])
def test_pieces_of_every_size(dim):
    """Sequences of one to many tiles of states in one call, so that pieces of one visit follow
    ones of many, in pairs and alone."""
    gen = torch.Generator(device="cuda").manual_seed(dim)
    sizes = [1, 130, 1, 1, 700, 127, 128, 129, 0, 3000, 2, 255, 257, 40, 511] * 4
    tokens = [33, 1, 2, 64, 31, 32, 5, 97, 3, 40, 1, 1, 130, 20, 7] * 4
    begin = torch.tensor([0] + sizes).cumsum(0)
    spans = torch.cat([torch.tensor([[int(b), int(b) + n]]).expand(t, 2) for b, n, t in zip(begin, sizes, tokens)]).int().cuda()
    T, S = spans.shape[0], int(begin[-1])
    q, k, v = _rand(gen, T, 8, dim), _rand(gen, S, 2, dim), _rand(gen, S, 2, dim)
    _check(q, k, v, spans)
