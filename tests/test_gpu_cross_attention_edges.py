"""Cross attention where its schedule and its numbers end, against the formulas in 64 bits
(those of test_gpu_cross_attention, with its tolerances)."""
import numpy as np
import pytest
import torch

import s3d8_a8_linear_gb300 as s3d8
from test_gpu_cross_attention import BF, _check, _lib, _rand, _reference, _within, _within_lse  # noqa: F401

pytestmark = pytest.mark.gpu

TILE = 128


# ---- pieces of one visit behind longer ones ---------------------------------


def _pieces(spans, S, heads, group, ctas):
    """How the forward pass divides its work, replayed: for each CTA its pieces, as (whether two
    query tiles go together, visits)."""
    each = TILE // group
    spans = [(max(a, 0), min(b, S)) if a < b else (0, 0) for a, b in spans.tolist()]
    tiles = -(-len(spans) // each)
    seen = [[(a // TILE, -(-b // TILE)) for a, b in spans[i * each:(i + 1) * each] if a < b] for i in range(tiles)]
    ends = [(min(a for a, _ in s), max(b for _, b in s)) if s else (0, 1) for s in seen]
    items = []
    for i in range(0, tiles, 2):
        both = ends[i:i + 2]
        if len(both) == 2 and 8 * (max(b for _, b in both) - min(a for a, _ in both)) <= 5 * sum(b - a for a, b in both) + 8:
            items.append((True, seen[i] + seen[i + 1]))
        else:
            items += [(False, s) for s in seen[i:i + 2]]
    sizes = [max(len({j for a, b in s for j in range(a, b)}), 1) for _, s in items]
    begin, total = np.cumsum([0] + sizes * heads), heads * sum(sizes)
    used, shares = min(total, ctas), []
    for c in range(used):
        at, end, share = total * c // used, total * (c + 1) // used, []
        while at < end:
            k = int(np.searchsorted(begin, at, "right")) - 1
            n = min(end, int(begin[k + 1])) - at
            share.append((items[k % len(items)][0], n))
            at += n
        shares.append(share)
    return shares


@pytest.mark.parametrize("T,most,dim,seeds", [(65, 1601, 128, (4, 5)), (97, 700, 128, (0, 1)), (33, 1601, 64, (1, 20))])
def test_pieces_of_one_visit(T, most, dim, seeds):
    """Batches of single tokens whose shares have a piece of one visit, in which the second of a
    CTA's two chains has nothing to do, right behind a longer one, whose two chains are joined."""
    ctas = torch.cuda.get_device_properties(0).multi_processor_count
    for seed in seeds:
        sizes = np.random.default_rng(seed).integers(0, most + 1, T)
        ends = np.cumsum(sizes)
        spans = torch.from_numpy(np.stack((ends - sizes, ends), -1).astype(np.int32)).cuda()
        S = int(ends[-1])
        shares = _pieces(spans, S, 8, 4, ctas)
        if ctas == 152:
            assert any(not a[0] and a[1] > 1 and b == (False, 1) for s in shares for a, b in zip(s, s[1:]))
        gen = torch.Generator(device="cuda").manual_seed(seed)
        q, k, v = _rand(gen, T, 32, dim), _rand(gen, S, 8, dim), _rand(gen, S, 8, dim)
        got = _check(q, k, v, spans, back=False)
        out, lse = torch.empty_like(got["out"]), torch.empty_like(got["lse"])
        for _ in range(200):
            s3d8.cross_attention(q, k, v, spans, out=out, lse=lse)
            assert torch.equal(out, got["out"]) and torch.equal(lse, got["lse"])


# ---- numbers at the ends of their range -------------------------------------


@pytest.mark.parametrize("T,S", [(1, 100), (1, 300), (1, 20000), (3, 130), (40, 9000), (70, 500)])
def test_scores_of_minus_infinity(T, S):
    """A token whose scores are all -infinity gets zeros and lse = -infinity, whether one piece of
    the work or several make its output; one that has others gets what those give."""
    gen = torch.Generator(device="cuda").manual_seed(S)
    q, k, v = _rand(gen, T, 4, 64), _rand(gen, S, 1, 64), _rand(gen, S, 1, 64)
    q[..., 0] = 1.0
    k[..., 0] = -float("inf")
    lse = torch.empty((T, 4), device="cuda")
    out = s3d8.cross_attention(q, k, v, lse=lse)
    assert not out.any() and (lse == -float("inf")).all()
    k[S // 2:, :, 0] = 0.5
    out = s3d8.cross_attention(q, k, v, lse=lse)
    r = _reference(q, k[S // 2:], v[S // 2:], None, 64 ** -0.5)
    _within(out, r["out"], r["out_tol"], "out")
    _within_lse(lse, r["lse"])


@pytest.mark.parametrize("scale,size", [(0.0, 2.0 ** 60), (2.0 ** -110, 2.0 ** 52), (-2.0 ** -110, 2.0 ** 52), (2.0 ** -60, 2.0 ** 30)])
def test_small_scales_of_large_products(scale, size):
    gen = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = _rand(gen, 40, 4, 64) * size, _rand(gen, 300, 2, 64) * size, _rand(gen, 300, 2, 64)
    _check(q, k, v, None, scale)


def test_spans_of_no_states_are_recorded():
    """Without states every span that is not empty leaves them."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    q, none = _rand(gen, 5, 4, 64), torch.empty((0, 2, 64), dtype=BF, device="cuda")
    lse = torch.empty((5, 4), device="cuda")
    spans = torch.tensor([[0, 0], [3, 3], [9, 2], [0, 0], [-4, -4]], device="cuda").int()
    out = s3d8.cross_attention(q, none, none, spans, lse=lse)
    g = s3d8.cross_attention_backward(q, q, none, none, out, lse, spans)
    assert s3d8.device_status() == 0
    assert not out.any() and not g["dq"].any() and (lse == -float("inf")).all()
    for bad in ([0, 1], [-3, 0], [5, 9]):
        spans[3] = torch.tensor(bad, device="cuda")
        out = s3d8.cross_attention(q, none, none, spans, lse=lse)
        assert s3d8.device_status() == -7 and not out.any() and (lse == -float("inf")).all()
        g = s3d8.cross_attention_backward(q, q, none, none, out, lse, spans)
        assert s3d8.device_status() == -7 and not g["dq"].any()


# ---- gradients ----------------------------------------------------------------


def test_what_an_infinity_reaches():
    """Infinities and NaN that tokens do see reach no gradient past the 128 query rows (here 64
    tokens) and the 128 states of the tiles that those tokens and states are in."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    T, S = 400, 1000
    q, k, v, dout = _rand(gen, T, 4, 64), _rand(gen, S, 2, 64), _rand(gen, S, 2, 64), _rand(gen, T, 4, 64)
    image = torch.arange(T, device="cuda") // 100
    spans = torch.stack((image * 250, image * 250 + 250), -1).int()
    lse = torch.empty((T, 4), device="cuda")

    def gradients():
        out = s3d8.cross_attention(q, k, v, spans, lse=lse)
        return s3d8.cross_attention_backward(dout, q, k, v, out, lse, spans)

    clean = gradients()
    tokens, states = torch.ones(T, dtype=torch.bool, device="cuda"), torch.ones(S, dtype=torch.bool, device="cuda")
    tokens[64:256], states[128:512] = False, False      # tiles with tokens 100 .. 199, with states 250 .. 499
    for t, j, bad in ((q, 150, float("nan")), (dout, 101, float("inf")), (k, 300, -float("inf")), (v, 499, float("nan")), (k, 250, float("inf"))):
        kept = t[j].clone()
        t[j] = bad
        got = gradients()
        t[j] = kept
        assert torch.equal(got["dq"][tokens], clean["dq"][tokens])
        assert all(torch.equal(got[n][states], clean[n][states]) for n in ("dk", "dv"))


def test_gradients_of_far_states():
    """Offsets past 2^31 elements, in keys and values and in their gradients."""
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    S, dim = (1 << 24) - 5, 128
    both = torch.empty((S, 4, dim), dtype=BF, device="cuda")        # 8.6 billion elements
    gen = torch.Generator(device="cuda").manual_seed(15)
    both[-700:] = _rand(gen, 700, 4, dim)
    both[:300] = _rand(gen, 300, 4, dim)
    q, dout = _rand(gen, 6, 4, dim), _rand(gen, 6, 4, dim)
    spans = torch.tensor([[S - 700, S], [S - 300, S - 1], [0, 300], [S - 30, S], [0, 100], [S - 40, S - 39]], device="cuda").int()
    near = torch.cat((both[:300], both[-700:]))
    moved = torch.where(spans >= 1000, spans - (S - 1000), spans)
    lse = torch.empty((6, 4), device="cuda")
    out = s3d8.cross_attention(q, both[:, :2], both[:, 2:], spans, lse=lse)
    g = s3d8.cross_attention_backward(dout, q, both[:, :2], both[:, 2:], out, lse, spans)
    r = _reference(q, near[:, :2], near[:, 2:], moved, dim ** -0.5, dout, out)
    _within(g["dq"], r["dq"], r["dq_tol"], "dq")
    for n in ("dk", "dv"):
        got = torch.cat((g[n][:300], g[n][-700:]))
        _within(got, r[n], r[n + "_tol"], n)
        assert not any(bool(part.any()) for part in g[n][300:-700].split(1 << 20)), n


@pytest.mark.parametrize("T,S,Hq,heads,dim", [(150, 5000, 2, 2, 128), (150, 5000, 4, 1, 40), (60, 2000, 128, 1, 8), (33, 700, 10, 2, 96), (90, 20, 3, 1, 64)])
def test_few_states_and_many_side_by_side(T, S, Hq, heads, dim):
    """Tokens of no, one, few and more than 128 states in one tile, in any order and far apart: the
    ones of at most 128 have delta from its parts."""
    gen = torch.Generator(device="cuda").manual_seed(dim)
    n = torch.tensor([0, 1, 2, 15, 16, 17, 100, 127, 128, 129, 130, 300], device="cuda")[torch.randint(0, 12, (T,), generator=gen, device="cuda")]
    lo = (torch.rand(T, generator=gen, device="cuda") * S).long()
    spans = torch.stack((lo, (lo + n).clamp(max=S)), -1).int()
    _check(_rand(gen, T, Hq, dim), _rand(gen, S, heads, dim), _rand(gen, S, heads, dim), spans)
