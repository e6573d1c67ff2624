"""The paged cache: rotary append, attention of one new token, and page calls,
against plain 64-bit (or whole-number) versions of their definitions.

Tolerances.  Attention: the output's bf16 rounding is at most 2^-9 of its size;
a score s is an fp32 sum of at most 256 products, off by at most about 2^-20 of
the largest score S, which moves its weight by as much, and weights enter the
second product with 16 bits or more: 2^-8 |ref| + (1e-4 + 2^-19 S) max |v|.  The
log-sum-exp is good to 1e-4 + 2^-19 S.  Append: one rounding to bf16 (2^-8 |ref| + 1e-6),
or to a code of scale s (s / 2, and 2^-8 |ref| + 1e-6 for the fp32 arithmetic).
"""
import math

import numpy as np
import pytest
import torch

import s3d8_a8_linear_gb300 as s3d8
from gpu_util import bf16_to_f64, dev

pytestmark = pytest.mark.gpu

BF, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    s3d8.load(build_if_missing=True)
    torch.cuda.set_device(0)
    yield
    assert s3d8.device_status() == 0


def _i32(a):
    return torch.tensor(a, dtype=I32, device=dev())


def _rand(g, *shape):
    return torch.randn(shape, generator=g).to(BF).to(dev())


def _cache(pages, page, heads, dim, int8, order, fill=float("nan")):
    """A cache in one of three memory orders, filled with what must never matter."""
    dt = torch.int8 if int8 else BF

    def make(dtype, cols, value):
        shape = {"head": (pages, heads, page), "token": (pages, page, heads), "mixed": (heads, page, pages)}[order]
        t = torch.full((*shape, *cols), value, dtype=dtype, device=dev())
        if order == "head":
            return t.transpose(1, 2)
        return t if order == "token" else t.permute(2, 1, 0, *range(3, 3 + len(cols)))

    kv = [make(dt, (dim,), 77 if int8 else fill) for _ in "kv"]
    return s3d8.KVCache(*kv, *([make(torch.float32, (), fill) for _ in "kv"] if int8 else []))


def _fill(cache, g, lens, width, page):
    """Random tokens for `lens` on scattered pages; returns the table, and the
    tokens' keys and values in 64 bits per row [n, heads, dim]."""
    used = [-(-n // page) for n in lens]
    order = torch.randperm(cache.pages, generator=g)
    table = torch.full((len(lens), width), -1, dtype=I32)
    rows, at = [], 0
    for b, n in enumerate(lens):
        ids = order[at:at + used[b]]
        at += used[b]
        table[b, :used[b]] = ids.to(I32)
        pos = torch.arange(n)
        p, t = ids[pos // page].to(dev()) if n else pos.to(dev()), (pos % page).to(dev())
        kv = []
        for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
            if s is None:
                x = _rand(g, n, cache.heads, cache.dim)
                c[p, t] = x
                kv.append(bf16_to_f64(x))
            else:
                x = torch.randint(-127, 128, (n, cache.heads, cache.dim), generator=g).to(torch.int8).to(dev())
                sc = (torch.rand((n, cache.heads), generator=g) * 0.03 + 1e-3).to(dev())
                c[p, t], s[p, t] = x, sc
                kv.append(x.cpu().numpy().astype(np.float64) * sc.double().cpu().numpy()[..., None])
        rows.append(kv)
    return table.to(dev()), rows


def _attend(q, k, v, scale, window, most=None):
    """64-bit attention of q [Hq, D] over k, v [n, H, D]; output and log-sum-exp
    (and the largest score's size, into the list `most`)."""
    n, H, D = k.shape
    if window:
        k, v = k[max(0, n - window):], v[max(0, n - window):]
    out, lse = np.zeros((q.shape[0], D)), np.full(q.shape[0], -math.inf)
    if not n:
        return out, lse
    G = q.shape[0] // H
    for h in range(q.shape[0]):
        s = k[:, h // G] @ q[h] * scale
        top = s.max()
        if most is not None:
            most.append(np.abs(s).max())
        p = np.exp(s - top)
        out[h], lse[h] = (p @ v[:, h // G]) / p.sum(), top + math.log(p.sum())
    return out, lse


def _check_attention(lens, heads, group, dim, page, int8=False, order="head", window=0, scale=None, seed=0,
                     workspace=None, width=None):
    g = torch.Generator().manual_seed(seed)
    width = max(1, max(-(-n // page) for n in lens)) + 1 if width is None else width
    cache = _cache(sum(-(-n // page) for n in lens) + 2, page, heads, dim, int8, order)
    table, rows = _fill(cache, g, lens, width, page)
    q = _rand(g, len(lens), heads * group, dim)
    lse = torch.full((len(lens), heads * group), 9.0, device=dev())
    out = s3d8.paged_attention(q, cache, table, _i32(lens), scale=scale, window=window, lse=lse, workspace=workspace)
    torch.cuda.synchronize()
    got, got_lse, qf = bf16_to_f64(out), lse.double().cpu().numpy(), bf16_to_f64(q)
    for b, (k, v) in enumerate(rows):
        most = [0.0]
        ref, ref_lse = _attend(qf[b], k, v, dim ** -0.5 if scale is None else scale, window, most)
        slack = 1e-4 + 2.0 ** -19 * max(most)
        tol = 2.0 ** -8 * np.abs(ref) + slack * (np.abs(v).max() if v.size else 0.0)
        assert (np.abs(got[b] - ref) <= tol).all(), (b, lens[b], np.abs(got[b] - ref).max())
        fine = np.isfinite(ref_lse)
        assert np.array_equal(fine, np.isfinite(got_lse[b])), (b, got_lse[b])
        assert (np.abs(got_lse[b][fine] - ref_lse[fine]) <= slack).all(), (b, lens[b])
    return out


LENS = [0, 1, 2, 15, 16, 17, 31, 33, 64, 129, 500]


@pytest.mark.parametrize("page", [16, 12])
@pytest.mark.parametrize("int8", [False, True])
def test_keys_and_values_of_unlike_strides(int8, page):
    """Keys with the heads outside, values with the tokens outside: append into them,
    attend over them, copy their pages."""
    g = torch.Generator().manual_seed(31)
    T, pages = 3 * page + 1, 9
    a, b = _cache(pages, page, 2, 64, int8, "head", fill=0.0), _cache(pages, page, 2, 64, int8, "token", fill=0.0)
    cache = s3d8.KVCache(a.k, b.v, a.k_scale, a.v_scale)
    table, none = _i32([[5, 2, 7, 0]]), torch.empty((64, 0), device=dev())
    q, k, v = (_rand(g, T, h, 64) for h in (8, 2, 2))
    s3d8.rope_append(q, k, v, none, none, _i32(range(T)), cache, table, rows=_i32([0] * T))
    s3d8.copy_pages(s3d8.KVPool([cache]), _i32([5, 2, 7, 0]), _i32([1, 3, 4, 8]))
    at = _i32([[1, 3, 4, 8]])
    pos = torch.arange(T, device=dev())
    where = at[0].long()[pos // page], pos % page
    kk, vv = (bf16_to_f64(c[where]) if sc is None else c[where].cpu().numpy() * sc[where].double().cpu().numpy()[..., None]
              for c, sc in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
    for new, have in ((k, kk), (v, vv)):
        new = bf16_to_f64(new)
        step = np.abs(new).max(-1, keepdims=True) / 127 if int8 else 0.0
        assert (np.abs(have - new) <= 0.5 * step + 2.0 ** -8 * np.abs(new) + 1e-6).all()
    got = bf16_to_f64(s3d8.paged_attention(q[:1].contiguous(), cache, at, _i32([T])))
    ref, _ = _attend(bf16_to_f64(q)[0], kk, vv, 0.125, 0)
    assert (np.abs(got[0] - ref) <= 2.0 ** -8 * np.abs(ref) + 1e-4 * np.abs(vv).max()).all()


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("dim,group", [(64, 1), (64, 12), (80, 4), (128, 4), (128, 12), (256, 4), (256, 16)])
def test_attention_shares_with_short_runs(dim, group, int8):
    """Enough tokens that every warp's share is cut into a long run and short ones."""
    lens = [40001, 3, 0, 77777, 12345]
    first = _check_attention(lens, 8, group, dim, 16, int8, seed=7)
    assert torch.equal(first, _check_attention(lens, 8, group, dim, 16, int8, seed=7))


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("group", [1, 3, 4, 7, 8, 9, 16, 17, 40])
def test_attention_groups(group, int8):
    _check_attention(LENS, 2, group, 64, 16, int8, seed=group)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("dim", [16, 32, 48, 64, 80, 112, 128, 144, 192, 240, 256])
def test_attention_dims(dim, int8):
    _check_attention(LENS, 3, 4, dim, 8, int8, "token", seed=dim)


@pytest.mark.parametrize("order", ["head", "token", "mixed"])
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("page", [1, 3, 8, 16, 24, 100, 256])
def test_attention_pages_and_orders(page, int8, order):
    _check_attention(LENS, 2, 4, 128, page, int8, order, seed=page)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("window", [1, 2, 16, 17, 100, 499, 500, 4096])
def test_attention_windows(window, int8):
    _check_attention(LENS, 2, 4, 128, 24, int8, window=window, seed=window)


@pytest.mark.parametrize("heads,group,lens,page", [
    (1, 8, [20000], 16),                      # one row over many CTAs
    (8, 4, [1] * 700, 4),                     # many rows of one token
    (2, 16, [0, 9000, 0, 0, 3, 4001, 0], 64),  # idle rows between long ones
    (8, 1, [0, 0, 0], 16),                    # nothing to read at all
    (4, 2, list(range(300)), 8),              # every length
    (1, 71, [333, 5000], 16),
])
@pytest.mark.parametrize("int8", [False, True])
def test_attention_splits(heads, group, lens, page, int8):
    first = _check_attention(lens, heads, group, 128, page, int8, seed=5)
    again = _check_attention(lens, heads, group, 128, page, int8, seed=5)
    assert torch.equal(first, again)          # the joins run in a fixed order


def test_attention_workspace_is_reused_whatever_it_holds():
    probe = _cache(4, 16, 2, 128, False, "head")
    ws = s3d8.paged_attention_workspace(probe, 16, 8)
    for value in (0, 255, 1, 128):
        ws.fill_(value)
        for lens in ([4000, 1, 0, 77] * 4, [5], [9000] * 3 + [1] * 13):
            _check_attention(lens, 2, 4, 128, 16, seed=value, workspace=ws)


def test_attention_extreme_scores():
    """Scores far beyond exp's range, and a scale of its own: the running maximum
    must carry them; lengths over several splits."""
    _check_attention([700, 3000, 1], 2, 4, 128, 16, scale=40.0)
    _check_attention([700, 3000, 1], 2, 4, 128, 16, True, scale=9.0)
    _check_attention([300, 2], 2, 4, 128, 16, scale=0.0)
    _check_attention([300, 2], 2, 4, 128, 16, scale=-0.5)


def test_attention_int8_scales_of_all_sizes():
    """Values whose scales differ by many orders, the largest on the weakest keys."""
    g = torch.Generator().manual_seed(2)
    lens, page = [513, 40], 16
    cache = _cache(60, page, 2, 128, True, "head")
    table, rows = _fill(cache, g, lens, 40, page)
    q = _rand(g, 2, 8, 128)
    for b, n in enumerate(lens):
        pos = torch.arange(n, device=dev())
        p, t = table[b].long()[pos // page], pos % page
        sc = (10.0 ** (torch.rand((n, 2), generator=g) * 16 - 12)).to(dev())
        cache.v_scale[p, t] = sc
        code = cache.v[p, t].cpu().numpy().astype(np.float64)
        rows[b][1] = code * sc.double().cpu().numpy()[..., None]
    out = bf16_to_f64(s3d8.paged_attention(q, cache, table, _i32(lens)))
    for b, (k, v) in enumerate(rows):
        ref, _ = _attend(bf16_to_f64(q)[b], k, v, 128 ** -0.5, 0)
        size, _ = _attend(bf16_to_f64(q)[b], k, np.abs(v), 128 ** -0.5, 0)
        assert (np.abs(out[b] - ref) <= 2.0 ** -8 * np.abs(ref) + 1e-4 * size).all()


def test_attention_nonfinite_values_reach_the_output():
    g = torch.Generator().manual_seed(3)
    cache = _cache(8, 16, 1, 64, False, "head")
    table, _ = _fill(cache, g, [40], 4, 16)
    q = _rand(g, 1, 4, 64)
    cache.v[table[0, 1].long(), 3, 0, 5] = float("nan")
    out = s3d8.paged_attention(q, cache, table, _i32([40]))
    bad = torch.isnan(out).cpu()
    assert bool(bad[:, :, 5].all()) and int(bad.sum()) == 4


def test_attention_long_offsets():
    """Pages beyond 2^31 elements from the cache's start."""
    pages = 140000
    k = torch.empty((pages, 16, 8, 128), dtype=BF, device=dev())
    v = torch.empty_like(k)
    g = torch.Generator().manual_seed(9)
    ids = torch.tensor([139999, 0, 131072, 135000, 131071, 7, 138888], device=dev())
    for c in (k, v):
        c[ids] = _rand(g, len(ids), 16, 8, 128)
    cache = s3d8.KVCache(k, v)
    q = _rand(g, 1, 32, 128)
    out = s3d8.paged_attention(q, cache, ids.to(I32)[None].contiguous(), _i32([105]))
    kk, vv = (bf16_to_f64(c[ids].reshape(-1, 8, 128)[:105]) for c in (k, v))
    ref, _ = _attend(bf16_to_f64(q)[0], kk, vv, 128 ** -0.5, 0)
    assert (np.abs(bf16_to_f64(out)[0] - ref) <= 2.0 ** -8 * np.abs(ref) + 1e-4 * np.abs(vv).max()).all()


def test_attention_on_another_stream():
    g = torch.Generator().manual_seed(4)
    cache = _cache(300, 16, 8, 128, False, "head")
    table, rows = _fill(cache, g, [4000], 256, 16)
    q = _rand(g, 1, 32, 128)
    want = s3d8.paged_attention(q, cache, table, _i32([4000]))
    lens = _i32([4000])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        mine = torch.zeros_like(q)
        for _ in range(50):          # q comes out of work queued on this stream
            mine.copy_(q)
        got = s3d8.paged_attention(mine, cache, table, lens)
    side.synchronize()
    assert torch.equal(got, want)


def test_attention_bad_pages_are_masked_and_recorded():
    g = torch.Generator().manual_seed(6)
    cache = _cache(8, 16, 1, 64, False, "head")
    table, rows = _fill(cache, g, [64, 40], 4, 16)
    table[0, 1], table[1, 0] = 8, -5
    q = _rand(g, 2, 4, 64)
    assert s3d8.device_status() == 0
    out = bf16_to_f64(s3d8.paged_attention(q, cache, table, _i32([64, 40])))
    assert s3d8.device_status() == -7 and s3d8.device_status() == 0
    for b, keep in ((0, [*range(16), *range(32, 64)]), (1, [*range(16, 40)])):
        ref, _ = _attend(bf16_to_f64(q)[b], rows[b][0][keep], rows[b][1][keep], 0.125, 0)
        assert (np.abs(out[b] - ref) <= 2.0 ** -8 * np.abs(ref) + 4e-4).all()
    ok = s3d8.paged_attention(q[:1], cache, _i32([[3, 4]]), _i32([0]))
    assert bool((ok == 0).all())
    table[0] = 99                                  # not one page to read
    out = s3d8.paged_attention(q, cache, table, _i32([64, -3]))
    assert bool((out == 0).all()) and s3d8.device_status() == -7
    s3d8.paged_attention(q[:1], cache, _i32([[0]]), _i32([17]))      # longer than its table
    assert s3d8.device_status() == -7


def test_attention_refusals():
    cache = _cache(8, 16, 2, 64, False, "head")
    q, table, lens = torch.zeros((1, 8, 64), dtype=BF, device=dev()), _i32([[0]]), _i32([3])
    with pytest.raises(ValueError):
        s3d8.paged_attention(q[..., :32].contiguous(), cache, table, lens)
    with pytest.raises(TypeError):
        s3d8.paged_attention(q.float(), cache, table, lens)
    with pytest.raises(TypeError):
        s3d8.paged_attention(q, cache, table.long(), lens)
    with pytest.raises(ValueError):
        s3d8.paged_attention(q, cache, _i32([[0], [1]]), lens)
    for bad in (dict(window=-1), dict(q=torch.zeros((1, 3, 64), dtype=BF, device=dev()))):
        with pytest.raises(s3d8.S3D8Error) as e:
            s3d8.paged_attention(**{**dict(q=q, cache=cache, table=table, lens=lens), **bad})
        assert e.value.status == -1
    with pytest.raises(s3d8.S3D8Error) as e:
        s3d8.paged_attention(q, cache, table, lens, workspace=torch.empty((8,), dtype=torch.uint8, device=dev()))
    assert e.value.status == -6
    with pytest.raises(ValueError):
        s3d8.KVCache(torch.zeros((2, 4, 1, 24), dtype=BF, device=dev()), torch.zeros((2, 4, 1, 24), dtype=BF, device=dev()))
    with pytest.raises(ValueError):
        s3d8.KVCache(cache.k.to(torch.int8), cache.v.to(torch.int8))
    with pytest.raises(TypeError):
        s3d8.KVCache(cache.k.half(), cache.v.half())
    with pytest.raises(ValueError):
        s3d8.KVCache(cache.k.transpose(2, 3), cache.v.transpose(2, 3))
    odd, odd2 = (torch.zeros((2, 16, 1, 68), dtype=BF, device=dev())[..., :64] for _ in "kv")   # rows of 136 bytes
    with pytest.raises(s3d8.S3D8Error) as e:
        s3d8.paged_attention(q, s3d8.KVCache(odd, odd2), table, lens)
    assert e.value.status == -2
    empty = s3d8.paged_attention(q[:0], cache, table[:0], lens[:0])
    assert empty.shape == (0, 8, 64)


# ---- append -----------------------------------------------------------------


def _turn(x, cos, sin, rotary, interleaved):
    x = x.copy()
    c, s = cos[:, None], sin[:, None]
    i = (slice(0, rotary, 2), slice(1, rotary, 2)) if interleaved else (slice(0, rotary // 2), slice(rotary // 2, rotary))
    a, b = x[..., i[0]].copy(), x[..., i[1]].copy()
    x[..., i[0]], x[..., i[1]] = a * c - b * s, b * c + a * s
    return x


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("heads,group,dim,rotary,page,order", [
    (8, 4, 128, 128, 16, "head"), (1, 7, 64, 64, 1, "token"), (2, 1, 80, 40, 24, "mixed"), (3, 2, 256, 128, 7, "head"),
    (2, 4, 16, 2, 8, "token"), (2, 2, 48, 22, 16, "head"), (2, 2, 96, 0, 16, "head"), (1, 1, 144, 18, 5, "token"),
])
def test_append(heads, group, dim, rotary, page, order, int8, interleaved):
    g = torch.Generator().manual_seed(dim + rotary)
    T, n_rows, width, max_pos = 67, 5, 40 // page + 2, 45
    cache = _cache(n_rows * width, page, heads, dim, int8, order, fill=-1.0)
    before = [t.clone() for t in (cache.k, cache.v)]
    table = torch.randperm(n_rows * width, generator=g).to(I32).view(n_rows, width).to(dev())
    place = torch.randperm(n_rows * 40, generator=g)[:T]
    rows, pos = (place // 40).to(I32), (place % 40).to(I32)
    pos[5] = pos[66] = -1 - 3          # padding
    fused = _rand(g, T, heads * group + 2 * heads, dim)      # q, k, v as slices of one projection
    q, k, v = fused[:, :heads * group], fused[:, heads * group:-heads], fused[:, -heads:]
    angle = torch.rand((max_pos, rotary // 2), generator=g) * 6
    cos, sin = angle.cos().to(dev()), angle.sin().to(dev())
    out = torch.full((T, heads * group, dim), 7.0, dtype=BF, device=dev())
    s3d8.rope_append(q, k, v, cos, sin, pos.to(dev()), cache, table, rows=rows.to(dev()), q_out=out,
                     interleaved=interleaved)
    torch.cuda.synchronize()
    real = pos >= 0
    c, s = (t.double().cpu().numpy()[pos.clamp(min=0).long()] for t in (cos, sin))
    ref = _turn(bf16_to_f64(q), c, s, rotary, interleaved) * real.numpy()[:, None, None]
    got = bf16_to_f64(out)
    assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 1e-6).all()
    where = (table.cpu()[rows.long(), (pos.clamp(min=0) // page).long()].long(), (pos.clamp(min=0) % page).long())
    touched = torch.zeros(cache.k.shape[:2], dtype=torch.bool)
    touched[where[0][real], where[1][real]] = True
    for i, (store, sc, new) in enumerate(((cache.k, cache.k_scale, _turn(bf16_to_f64(k), c, s, rotary, interleaved)),
                                          (cache.v, cache.v_scale, bf16_to_f64(v)))):
        new = new[real.numpy()]
        at = (where[0][real].to(dev()), where[1][real].to(dev()))
        have = store[at].double().cpu().numpy()
        tol = 2.0 ** -8 * np.abs(new) + 1e-6
        if int8:
            step = sc[at].double().cpu().numpy()[..., None]
            top = np.abs(new).max(-1, keepdims=True)
            assert (np.abs(step * 127 - top) <= 1e-6 * top + 1e-30).all()
            have, tol = have * step, 0.5 * step + 2.0 ** -8 * np.abs(new) + 1e-6
        assert (np.abs(have - new) <= tol).all(), np.abs(have - new).max()
        assert torch.equal(store.cpu()[~touched], before[i].cpu()[~touched])


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("T,heads,group,dim,rotary,interleaved,apart", [
    (305, 8, 4, 128, 128, False, False), (1500, 2, 4, 128, 64, False, True), (5003, 1, 1, 16, 16, True, False),
    (777, 2, 3, 48, 32, True, True), (640, 1, 8, 256, 0, False, False), (401, 3, 2, 80, 48, False, False),
    (350, 2, 2, 64, 22, False, False), (613, 16, 8, 256, 256, True, True),
])
def test_append_many_tokens(T, heads, group, dim, rotary, interleaved, apart, int8):
    """Many tokens at once: against the formula in 64 bits, with padding, positions past the
    table of angles, rows past the table of pages and pages that are not there among them;
    `apart`: heads of q that do not follow one another."""
    g = torch.Generator().manual_seed(T)
    page, n_rows, Hq = 16, 4, heads * group
    width = T // n_rows // page + 2
    max_pos = width * page - 5
    cache = _cache(n_rows * width, page, heads, dim, int8, "head", fill=-1.0)
    before = [t.clone() for t in (cache.k, cache.v)]
    table = torch.randperm(n_rows * width, generator=g).to(I32).view(n_rows, width)
    table[2, 1], table[3, 0] = n_rows * width, -1
    place = torch.randperm(n_rows * (T // n_rows + 1), generator=g)[:T]
    rows, pos = (place % n_rows).to(I32), (place // n_rows).to(I32)
    pos[7], pos[T - 1], pos[T // 2] = -1, -9, max_pos if rotary else width * page
    rows[11], rows[12] = n_rows, -1
    fused = _rand(g, T, Hq + 2 * heads, dim)
    q, k, v = fused[:, :Hq], fused[:, Hq:-heads], fused[:, -heads:]
    if apart:
        q = _rand(g, T, 2 * Hq, dim)[:, ::2]
    angle = torch.rand((max_pos, rotary // 2), generator=g) * 6
    cos, sin = angle.cos().to(dev()), angle.sin().to(dev())
    assert s3d8.device_status() == 0
    out = s3d8.rope_append(q, k, v, cos, sin, pos.to(dev()), cache, table.to(dev()), rows=rows.to(dev()),
                           interleaved=interleaved)
    assert s3d8.device_status() == -7
    real = (pos >= 0) & ((pos < max_pos) | (rotary == 0))
    col = pos.clamp(min=0).long() // page
    stored = real & (rows >= 0) & (rows < n_rows) & (col < width)
    pages = table[rows.clamp(0, n_rows - 1).long(), col.clamp(max=width - 1)].long()
    stored &= (pages >= 0) & (pages < n_rows * width)
    c, s = (t.double().cpu().numpy()[pos.clamp(0, max_pos - 1).long()] for t in (cos, sin))
    ref = _turn(bf16_to_f64(q), c, s, rotary, interleaved) * real.numpy()[:, None, None]
    assert (np.abs(bf16_to_f64(out) - ref) <= 2.0 ** -8 * np.abs(ref) + 1e-6).all()
    where = (pages[stored], pos[stored].long() % page)
    touched = torch.zeros(cache.k.shape[:2], dtype=torch.bool)
    touched[where] = True
    at = tuple(i.to(dev()) for i in where)
    for i, (store, sc, new) in enumerate(((cache.k, cache.k_scale, _turn(bf16_to_f64(k), c, s, rotary, interleaved)),
                                          (cache.v, cache.v_scale, bf16_to_f64(v)))):
        new = new[stored.numpy()]
        have = store[at].double().cpu().numpy()
        tol = 2.0 ** -8 * np.abs(new) + 1e-6
        if int8:
            step = sc[at].double().cpu().numpy()[..., None]
            top = np.abs(new).max(-1, keepdims=True)
            assert (np.abs(step * 127 - top) <= 1e-6 * top + 1e-30).all()
            have, tol = have * step, 0.5 * step + 2.0 ** -8 * np.abs(new) + 1e-6
        assert (np.abs(have - new) <= tol).all(), np.abs(have - new).max()
        assert torch.equal(store.cpu()[~touched], before[i].cpu()[~touched])


def test_append_then_attend_and_rows_default():
    """A decode step: token t of row t, then attention over it and what was there."""
    g = torch.Generator().manual_seed(21)
    lens, page = [5, 16, 33], 16
    cache = _cache(12, page, 2, 64, False, "head")
    table, rows = _fill(cache, g, lens, 4, page)
    table[1, 1] = 11 if 11 not in table.flatten().tolist() else int((set(range(12)) - set(table.flatten().tolist())).pop())
    q, k, v = (_rand(g, 3, h, 64) for h in (8, 2, 2))
    none = torch.empty((64, 0), device=dev())
    out = s3d8.rope_append(q, k, v, none, none, _i32(lens), cache, table)
    assert torch.equal(out, q)
    got = bf16_to_f64(s3d8.paged_attention(out, cache, table, _i32([n + 1 for n in lens])))
    for b in range(3):
        kk, vv = (np.concatenate([old, bf16_to_f64(new)[b][None]]) for old, new in zip(rows[b], (k, v)))
        ref, _ = _attend(bf16_to_f64(q)[b], kk, vv, 0.125, 0)
        assert (np.abs(got[b] - ref) <= 2.0 ** -8 * np.abs(ref) + 4e-4).all()


def test_append_out_of_range_is_skipped_and_recorded():
    g = torch.Generator().manual_seed(1)
    cache = _cache(4, 8, 1, 32, False, "head", fill=-1.0)
    table = _i32([[0, 9], [-1, 2]])
    q, k, v = (_rand(g, 6, 1, 32) for _ in range(3))
    cos = torch.ones((20, 16), device=dev())
    sin = torch.zeros_like(cos)
    pos, rows = _i32([3, 8, 0, 16, 20, 9]), _i32([0, 0, 1, 0, 0, 7])
    assert s3d8.device_status() == 0
    out = s3d8.rope_append(q, k, v, cos, sin, pos, cache, table, rows=rows)
    assert s3d8.device_status() == -7
    want = q.clone()
    want[4] = 0                                    # no table entry for its angle
    assert torch.equal(out, want)
    left = torch.full((4, 8, 1, 32), -1.0, dtype=BF, device=dev())
    left[0, 3] = k[0]
    assert torch.equal(cache.k, left)


def test_append_refusals():
    cache = _cache(4, 8, 1, 32, False, "head")
    z = torch.zeros((2, 1, 32), dtype=BF, device=dev())
    cos, pos, table = torch.zeros((8, 16), device=dev()), _i32([0, 1]), _i32([[0], [1]])
    with pytest.raises(ValueError):
        s3d8.rope_append(z, z[:1], z, cos, cos, pos, cache, table)
    with pytest.raises(ValueError):
        s3d8.rope_append(z, z, z, cos, cos[:4], pos, cache, table)
    with pytest.raises(TypeError):
        s3d8.rope_append(z, z, z, cos.double(), cos, pos, cache, table)
    with pytest.raises(TypeError):
        s3d8.rope_append(z, z, z, cos, cos, pos.long(), cache, table)
    wide = torch.zeros((8, 17), device=dev())
    with pytest.raises(s3d8.S3D8Error) as e:
        s3d8.rope_append(z, z, z, wide, wide, pos, cache, table)
    assert e.value.status == -1
    odd = torch.zeros((2, 1, 36), dtype=BF, device=dev())[..., 4:]
    with pytest.raises(s3d8.S3D8Error) as e:
        s3d8.rope_append(odd, z, z, cos, cos, pos, cache, table)
    assert e.value.status == -2
    assert s3d8.rope_append(z[:0], z[:0], z[:0], cos, cos, pos[:0], cache, table[:0]).shape == (0, 1, 32)


# ---- pages ------------------------------------------------------------------


class Plain:
    """The page calls on whole numbers, one entry after another."""

    def __init__(self, table, lens, refs, page):
        self.table, self.lens, self.refs, self.page = table.copy(), lens.copy(), refs.copy(), page

    def _take(self, need, state):
        ids = np.flatnonzero(self.refs == 0)[:need]
        if need and (state["full"] or len(ids) < need):
            state["full"] = True
            return None
        return ids

    def extend(self, seqs, add):
        got, state = [], {"full": False}
        for s, a in zip(seqs, add):
            have, want = -(-self.lens[s] // self.page), -(-(self.lens[s] + a) // self.page)
            ids = self._take(want - have, state) if want <= self.table.shape[1] else None
            got.append(int(ids is not None))
            if ids is not None:
                self.table[s, have:want] = ids
                self.refs[ids] = 1
                self.lens[s] += a
        return got

    def fork(self, parents, children):
        got, copies, state = [], [], {"full": False}
        for p, c in zip(parents, children):
            full, part = divmod(int(self.lens[p]), self.page)
            ids = self._take(int(part > 0), state)
            got.append(int(ids is not None))
            self.table[c], self.lens[c] = -1, 0
            if ids is None:
                continue
            self.table[c, :full] = self.table[p, :full]
            self.refs[self.table[p, :full]] += 1
            self.lens[c] = self.lens[p]
            if part:
                self.table[c, full] = ids[0]
                self.refs[ids[0]] = 1
                copies.append((int(self.table[p, full]), int(ids[0]), part))
        return got, copies

    def free(self, seqs):
        for s in seqs:
            for id in self.table[s][self.table[s] >= 0]:
                self.refs[id] -= 1
            self.table[s], self.lens[s] = -1, 0

    def compact(self):
        live = int((self.refs != 0).sum())
        holes = [i for i in range(live) if self.refs[i] == 0]
        movers = [i for i in range(live, len(self.refs)) if self.refs[i] != 0]
        for a, b in zip(movers, holes):
            self.table[self.table == a] = b
            self.refs[b], self.refs[a] = self.refs[a], 0
        return live, list(zip(movers, holes))


def _state(plain):
    return [_i32(x) for x in (plain.table, plain.lens, plain.refs)]


def _same(plain, table, lens, refs):
    assert np.array_equal(table.cpu().numpy(), plain.table)
    assert np.array_equal(lens.cpu().numpy(), plain.lens)
    assert np.array_equal(refs.cpu().numpy(), plain.refs)


def _pool(layers, pages, page, heads, dim, int8, order, seed):
    g = torch.Generator().manual_seed(seed)
    caches = []
    for _ in range(layers):
        c = _cache(pages, page, heads, dim, int8, order, fill=0.0)
        for t in (c.k, c.v, c.k_scale, c.v_scale):
            if t is not None:
                t.copy_(torch.randint(-100, 100, t.shape, generator=g).to(t.dtype))
        caches.append(c)
    return s3d8.KVPool(caches)


def _parts(pool):
    return [t for c in pool.caches for t in (c.k, c.v, c.k_scale, c.v_scale) if t is not None]


@pytest.mark.parametrize("order", ["head", "token", "mixed"])
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("layers,pages,page,heads,dim", [(1, 40, 8, 2, 64), (3, 33, 5, 3, 48), (70, 12, 16, 1, 16)])
def test_copy_pages(layers, pages, page, heads, dim, int8, order):
    pool = _pool(layers, pages, page, heads, dim, int8, order, 1)
    want = [t.clone() for t in _parts(pool)]
    src, dst = [0, 5, -1, 7, pages - 1, 2], [3, 4, 6, -1, 1, 10]
    s3d8.copy_pages(pool, _i32(src), _i32(dst))
    for t in want:
        for a, b in zip(src, dst):
            if a >= 0 and b >= 0:
                t[b] = t[a]
    assert all(torch.equal(a, b) for a, b in zip(_parts(pool), want))
    s3d8.copy_pages(pool, _i32([]), _i32([]))
    assert s3d8.device_status() == 0
    s3d8.copy_pages(pool, _i32([pages, 0]), _i32([1, pages]))
    assert s3d8.device_status() == -7
    assert all(torch.equal(a, b) for a, b in zip(_parts(pool), want))


@pytest.mark.parametrize("int8,order,pages,rows,width,page", [
    (False, "head", 64, 12, 9, 8), (True, "token", 200, 40, 12, 5), (False, "mixed", 1, 3, 2, 4),
    (False, "token", 5000, 1500, 4, 16), (True, "head", 40, 60, 3, 1),
])
def test_a_life_of_pages(int8, order, pages, rows, width, page):
    """Random growth, forks, release and compaction: tables, counts and every
    layer's contents after each call."""
    rng = np.random.default_rng(pages)
    pool = _pool(2, pages, page, 2, 32, int8, order, pages)
    plain = Plain(np.full((rows, width), -1, np.int32), np.zeros(rows, np.int32), np.zeros(pages, np.int32), page)
    table, lens, refs = _state(plain)
    ws = s3d8.pages_workspace(pool, rows)
    want = [t.clone() for t in _parts(pool)]
    for step in range(24):
        what = ["extend", "fork", "free", "compact"][step % 4]
        some = rng.permutation(rows)[:max(1, rows // 2)]
        ws.fill_(step * 37 % 256)
        if what == "extend":
            add = rng.integers(0, width * page // 2 + 2, len(some))
            got = s3d8.extend_pages(table, lens, refs, _i32(some), _i32(add), page, workspace=ws)
            assert got.tolist() == plain.extend(some, add)
        elif what == "fork":
            idle = np.flatnonzero(plain.lens == 0)
            busy = np.flatnonzero(plain.lens > 0)
            n = min(len(idle), 2 * len(busy))
            parents, children = (rng.choice(busy, n), rng.permutation(idle)[:n]) if n else ([], [])
            got = s3d8.fork_pages(pool, table, lens, refs, _i32(parents), _i32(children), workspace=ws)
            expect, copies = plain.fork(parents, children)
            assert got.tolist() == expect
            for a, b, tokens in copies:
                for t in want:
                    t[b, :tokens] = t[a, :tokens]
        elif what == "free":
            some = some[:max(1, rows // 3)]
            s3d8.free_pages(table, lens, refs, _i32(some))
            plain.free(some)
        else:
            live = s3d8.compact_pages(pool, table, refs, workspace=ws)
            expect, moves = plain.compact()
            assert live.tolist() == [expect]
            for a, b in moves:
                for t in want:
                    t[b] = t[a]
        _same(plain, table, lens, refs)
        assert all(torch.equal(a, b) for a, b in zip(_parts(pool), want)), (step, what)


def test_pages_bad_entries_are_refused_and_recorded():
    pool = _pool(1, 8, 4, 1, 16, False, "head", 0)
    plain = Plain(np.array([[0, 1, -1], [2, -1, -1], [-1, -1, -1]], np.int32), np.array([6, 4, 0], np.int32),
                  np.array([1, 1, 1, 0, 0, 0, 0, 0], np.int32), 4)
    table, lens, refs = _state(plain)
    assert s3d8.device_status() == 0
    assert s3d8.extend_pages(table, lens, refs, _i32([7, -1, 1]), _i32([1, 1, 3]), 4).tolist() == [0, 0, 1]
    assert s3d8.device_status() == -7
    plain.extend([1], [3])
    assert s3d8.extend_pages(table, lens, refs, _i32([0]), _i32([-2]), 4).tolist() == [0]
    _same(plain, table, lens, refs)
    assert s3d8.fork_pages(pool, table, lens, refs, _i32([9, 0]), _i32([2, 5])).tolist() == [0, 0]
    assert s3d8.device_status() == -7
    _same(plain, table, lens, refs)
    s3d8.free_pages(table, lens, refs, _i32([4]))
    assert s3d8.device_status() == -7
    refs[0] = 0                                  # counted by nobody, held by row 0
    s3d8.free_pages(table, lens, refs, _i32([0]))
    assert s3d8.device_status() == -7 and int(refs.min()) == 0
    assert s3d8.device_status() == 0


def test_pages_refusals():
    pool = _pool(1, 8, 4, 1, 16, False, "head", 0)
    table, lens, refs = _i32([[0, 1]]), _i32([6]), _i32([1, 1] + [0] * 6)
    with pytest.raises(ValueError):
        s3d8.fork_pages(pool, table, lens, refs[:4].clone(), _i32([0]), _i32([0]))
    with pytest.raises(ValueError):
        s3d8.extend_pages(table, _i32([1, 2]), refs, _i32([0]), _i32([1]), 4)
    with pytest.raises(TypeError):
        s3d8.free_pages(table.long(), lens, refs, _i32([0]))
    with pytest.raises(s3d8.S3D8Error) as e:        # more entries than rows
        s3d8.free_pages(table, lens, refs, _i32([0, 0]))
    assert e.value.status == -1
    with pytest.raises(s3d8.S3D8Error) as e:
        s3d8.compact_pages(pool, table, refs, workspace=torch.empty((8,), dtype=torch.uint8, device=dev()))
    assert e.value.status == -6
    with pytest.raises(s3d8.S3D8Error) as e:        # layers of unlike geometry
        s3d8.copy_pages(s3d8.KVPool([pool.caches[0], _cache(9, 4, 1, 16, False, "head")]), _i32([0]), _i32([1]))
    assert e.value.status == -1
    with pytest.raises(ValueError):
        s3d8.KVPool([])
