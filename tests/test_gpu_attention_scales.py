"""Attention over int8 caches whose value scales differ by many orders, against 64 bits.

Tolerance.  As in test_gpu_kv_cache: the output's rounding (2^-8 of its size, generously)
and the scores' (2^-19 of the largest score S moves a weight by as much).  A weight times
its value's scale enters the second product with 22 bits, or to 2^-30 of the largest one
that its query row meets, whichever is coarser: over n tokens with codes up to 127, n 127
2^-30 of that product, and the row's weighted size reaches about 127 times it in some
column, so n 2^-30 of the row's largest weighted size covers it.  All sizes are the
softmax-weighted ones, which tokens of no weight do not enter whatever their scale:
  2^-8 |ref| + (1e-4 + 2^-19 S) size + n 2^-30 max(size).
"""
import numpy as np
import pytest
import torch

import s3d8_a8_linear_gb300 as s3d8
from gpu_util import bf16_to_f64, dev
from test_gpu_kv_cache import _attend, _cache, _fill, _i32, _lib, _rand  # noqa: F401

pytestmark = pytest.mark.gpu


def _scores(q, k, scale, group):
    """[n, heads, group] of q [heads * group, dim] and k [n, heads, dim]."""
    return np.einsum("hgd,nhd->nhg", q.reshape(k.shape[1], group, -1), k) * scale


def _check(lens, heads, group, dim, page, scale, change, seed=0, window=0):
    """`change` gets the scores [n, heads, group] and the value scales [n, heads] of a sequence
    and returns new value scales."""
    g = torch.Generator().manual_seed(seed)
    width = max(-(-n // page) for n in lens) + 1
    cache = _cache(sum(-(-n // page) for n in lens) + 2, page, heads, dim, True, "head")
    table, rows = _fill(cache, g, lens, width, page)
    q = _rand(g, len(lens), heads * group, dim)
    qf = bf16_to_f64(q)
    for b, n in enumerate(lens):
        pos = torch.arange(n, device=dev())
        at = table[b].long()[pos // page], pos % page
        s = _scores(qf[b], rows[b][0], scale, group)
        sc = torch.from_numpy(change(s, cache.v_scale[at].double().cpu().numpy())).float().to(dev())
        cache.v_scale[at] = sc
        rows[b][1] = cache.v[at].cpu().numpy().astype(np.float64) * sc.double().cpu().numpy()[..., None]
    lse = torch.empty((len(lens), heads * group), device=dev())
    out = bf16_to_f64(s3d8.paged_attention(q, cache, table, _i32(lens), scale=scale, window=window, lse=lse))
    lse = lse.double().cpu().numpy()
    for b, (k, v) in enumerate(rows):
        most = [0.0]
        ref, ref_lse = _attend(qf[b], k, v, scale, window, most)
        size, _ = _attend(qf[b], k, np.abs(v), scale, window)
        slack = 1e-4 + 2.0 ** -19 * max(most)
        tol = 2.0 ** -8 * np.abs(ref) + slack * size + lens[b] * 2.0 ** -30 * size.max(-1, keepdims=True)
        off = np.abs(out[b] - ref) - tol
        assert (off <= 0).all(), (b, lens[b], (off / size.max(-1, keepdims=True)).max())
        assert (np.abs(lse[b] - ref_lse) <= slack).all()


def _outliers(ratio, gap=40.0):
    """In every 16 tokens, the one that every query of its head scores farthest below its top gets `ratio` times the
    scale, if that is at least `gap`."""
    def change(s, sc):
        sc, below = sc.copy(), (s.max(0, keepdims=True) - s).min(-1)      # [n, heads]
        put = 0
        for t in range(0, len(sc), 16):
            for h in range(sc.shape[1]):
                j = t + int(below[t:t + 16, h].argmax())
                if below[j, h] >= gap:
                    sc[j, h] *= ratio
                    put += 1
        assert put > sc.size // 64
        return sc
    return change


@pytest.mark.parametrize("ratio", [2.0 ** 20, 2.0 ** 24, 2.0 ** 27, 2.0 ** 31])
@pytest.mark.parametrize("heads,group,dim,page", [
    (2, 4, 128, 16), (2, 1, 64, 8), (8, 2, 256, 32), (2, 12, 128, 16), (1, 9, 64, 16), (1, 16, 256, 3), (3, 4, 80, 48),
])
def test_a_large_scale_on_a_token_of_no_weight_costs_nothing(heads, group, dim, page, ratio):
    _check([600, 4001, 17], heads, group, dim, page, 3.0 * 128 ** 0.5 / dim ** 0.5, _outliers(ratio), seed=dim + group)


@pytest.mark.parametrize("heads,group,dim", [(1, 4, 128), (1, 2, 64), (1, 4, 256), (1, 12, 128)])
def test_query_rows_that_look_at_values_of_unlike_scales(heads, group, dim):
    """The tokens that each second query looks at have scales 2^-24 of the others'."""
    def change(s, sc):
        sc, near = sc.copy(), s.max(0, keepdims=True) - s < 15.0         # [n, heads, group]
        small = near[..., ::2].any(-1) & ~near[..., 1::2].any(-1)
        assert small.any()
        sc[small] *= 2.0 ** -24
        return sc
    _check([700, 3000, 40], heads, group, dim, 16, 4.0 * 128 ** 0.5 / dim ** 0.5, change, seed=group)


def test_scales_at_both_ends_of_their_range():
    """All scales tiny, all huge, zeros between, and zeros up to the last tokens."""
    for factor in (1e-28, 1e28):
        _check([300, 50], 2, 4, 128, 16, 0.05, lambda s, sc: sc * factor)
        _check([300, 50], 2, 4, 128, 16, 0.05, lambda s, sc: sc * factor * (np.arange(len(sc)) % 3 == 0)[:, None])

    def late(s, sc):
        sc = sc.copy()
        sc[:-3] = 0.0
        return sc
    _check([300, 50, 4000], 2, 4, 128, 16, 0.05, late)
    _check([5000] * 40, 2, 4, 64, 16, 0.05, late)


def test_scales_next_to_the_largest_and_the_smallest():
    """Value scales up to 2^117 and down to 2^-120: outputs that bf16 still holds."""
    for factor in (4e36, 1e-34):
        _check([40, 17], 2, 4, 128, 16, 0.05, lambda s, sc: sc * factor)
        _check([40, 17], 2, 12, 64, 16, 0.05, lambda s, sc: sc * factor)


def test_scales_that_grow_along_the_sequence():
    def grow(s, sc):
        return sc * 2.0 ** (np.arange(len(sc)) * (60.0 / len(sc)) - 30)[:, None]
    for lens in ([900, 33], [3000] * 30):
        _check(lens, 2, 4, 128, 16, 0.05, grow)
        _check(lens, 2, 4, 128, 16, 0.05, lambda s, sc: grow(s, sc)[::-1].copy())


def test_nonfinite_scales_reach_only_their_own_rows():
    """A NaN value scale on a visible token makes its head's outputs NaN and no other's; a NaN key
    scale the log-sum-exp as well; behind the length or in front of the window neither matters."""
    g = torch.Generator().manual_seed(5)
    cache = _cache(40, 16, 2, 128, True, "head")
    table, _ = _fill(cache, g, [500], 33, 16)
    q = _rand(g, 1, 8, 128)
    want = s3d8.paged_attention(q, cache, table, _i32([500]), window=100)
    cache.v_scale[table[0, 3].long(), 2, 1] = float("nan")           # token 50
    lse = torch.empty((1, 8), device=dev())
    assert torch.equal(s3d8.paged_attention(q, cache, table, _i32([500]), window=100), want)
    out = s3d8.paged_attention(q, cache, table, _i32([500]), lse=lse)
    assert bool(torch.isnan(out[0, 4:]).all()) and bool(torch.isfinite(out[0, :4]).all()) and bool(torch.isfinite(lse).all())
    cache.k_scale[table[0, 3].long(), 2, 1] = float("nan")
    out = s3d8.paged_attention(q, cache, table, _i32([500]), lse=lse)
    assert bool(torch.isnan(out[0, 4:]).all()) and bool(torch.isnan(lse[0, 4:]).all()) and bool(torch.isfinite(lse[0, :4]).all())


@pytest.mark.parametrize("group", [4, 12])
def test_runs_of_tokens_whose_pages_are_not_there(group):
    """Long stretches of masked tokens, whole runs of them, before, between and behind visible ones."""
    g = torch.Generator().manual_seed(group)
    n, page = 40000, 16
    cache = _cache(n // page, page, 1, 128, True, "token")
    table, rows = _fill(cache, g, [n], n // page, page)
    q = _rand(g, 1, group, 128)
    pages = np.arange(n // page)
    for there in (pages % 700 == 650, pages == 0, pages == pages[-1], pages < 0):
        at = torch.where(torch.from_numpy(there).to(dev()), table[0], cache.pages)[None].contiguous()
        lse = torch.empty((1, group), device=dev())
        assert s3d8.device_status() == 0
        out = bf16_to_f64(s3d8.paged_attention(q, cache, at, _i32([n]), lse=lse))[0]
        assert s3d8.device_status() == -7
        keep = np.repeat(there, page)
        k, v = (x[keep] for x in rows[0])
        if not keep.any():
            assert (out == 0).all() and bool((lse == -float("inf")).all())
            continue
        most = [0.0]
        ref, ref_lse = _attend(bf16_to_f64(q)[0], k, v, 128 ** -0.5, 0, most)
        size, _ = _attend(bf16_to_f64(q)[0], k, np.abs(v), 128 ** -0.5, 0)
        slack = 1e-4 + 2.0 ** -19 * max(most)
        assert (np.abs(out - ref) <= 2.0 ** -8 * np.abs(ref) + slack * size + n * 2.0 ** -30 * size.max(-1, keepdims=True)).all()
        assert (np.abs(lse.double().cpu().numpy()[0] - ref_lse) <= slack).all()
