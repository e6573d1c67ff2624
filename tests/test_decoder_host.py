"""Host-side checks of the calls between two linears (no GPU): argument rejection
before any CUDA call, workspace sizes, and the binding's own checks.  Dummy
addresses are never dereferenced; they are passed only on a machine without a
CUDA device."""
import ctypes

import pytest
import torch

import s3d8_a8_linear_gb300 as s3d8
from s3d8_a8_linear_gb300 import _build
from s3d8_a8_linear_gb300.decoder import KVCacheStruct

no_device_only = pytest.mark.skipif(torch.cuda.is_available(),
                                    reason="dummy-pointer rejection tests run only without a GPU")

A, B, C, D = 0x10000, 0x20000, 0x30000, 0x40000


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return s3d8.load()


def _cache(**more):
    c = KVCacheStruct(k=A, v=B, pages=10, page_size=16, heads=2, dim=64, dtype=0)
    c.k_stride[:] = c.v_stride[:] = [2048, 128, 64]
    for name, value in more.items():
        if isinstance(value, list):
            getattr(c, name)[:] = value
        else:
            setattr(c, name, value)
    return c


@no_device_only
def test_residual_norm_rejects(lib):
    def f(h=A, y=B, wo=None, g=None, gn=0, wp=C, M=2, cols=64, ho=D, x=D, xq=None, xs=None):
        return lib.s3d8_residual_norm(h, y, wo, g, gn, 0, wp, 1.0, 1e-5, M, cols, ho, x, xq, xs, None)

    for cols in (0, 4, 12, -8, 16392):
        assert f(cols=cols) == -1, cols
    assert f(M=-1) == -1 and f(h=None) == -1 and f(y=None) == -1 and f(ho=None) == -1 and f(x=None) == -1
    assert f(g=A) == -1 and f(gn=1) == -1 and f(g=A, gn=7) == -1
    assert f(wp=None) == -1 and f(y=None, ho=None, wp=None, x=None) == -1
    assert f(xq=A, xs=A) == -1 and f(x=None, xq=A) == -1
    assert f(cols=72, x=None, xq=A, xs=A) == -1           # codes need rows of 16
    assert f(h=A + 2) == -2 and f(wp=C + 8) == -2 and f(g=A + 2, gn=64) == -2 and f(x=None, xq=A + 4, xs=A) == -2
    assert f(M=0, h=None, y=None, ho=None, x=None) == 0

    def b(dh=A, dx=A, h=A, y=B, wo=None, g=None, gn=0, wp=C, M=2, cols=64, dhi=D, dy=D, dwp=A, dwo=None, dg=None, ws=A,
          n=1 << 20):
        return lib.s3d8_residual_norm_backward(dh, dx, h, y, wo, g, gn, 0, wp, 1.0, 1e-5, M, cols, dhi, dy, dwp, dwo, dg,
                                               ws, n, None)

    assert b(dwp=None) == -1 and b(dwo=A) == -1 and b(dg=A) == -1 and b(wo=A) == -1 and b(dhi=None) == -1
    assert b(dy=None) == -1 and b(y=None) == -1 and b(wp=None, dwp=None) == -1 and b(cols=20) == -1
    assert b(ws=None) == -6 and b(n=4) == -6 and b(ws=A + 8) == -2 and b(dx=A + 4) == -2 and b(dwp=A + 4) == -2
    size = lib.s3d8_residual_norm_backward_workspace_size
    assert size(0, 64) == 0 and size(5, 12) == 0 and size(5, 64) >= 5 * 2 * 64 * 4


@no_device_only
def test_cache_geometry_is_checked(lib):
    def f(c, B=1, Hq=4, width=2, window=0, q=A, lens=A, out=A, ws=A, n=1 << 30, table=A):
        return lib.s3d8_paged_attention(q, ctypes.byref(c) if c else None, table, width, lens, B, Hq, 0.125, window, out, None,
                                        ws, n, None)

    assert f(None) == -1
    for bad in (dict(k=None), dict(v=None), dict(pages=0), dict(page_size=0), dict(heads=0), dict(dim=0), dict(dim=24),
                dict(dim=272), dict(dtype=2), dict(dtype=1), dict(pages=1 << 28), dict(k_stride=[-8, 128, 64])):
        assert f(_cache(**bad)) == -1, bad
    for bad in (dict(k=A + 8), dict(v=B + 2), dict(k_stride=[2048, 132, 64]),
                dict(dtype=1, k_scale=A, v_scale=A, k_stride=[2048, 128, 72]), dict(dtype=1, k_scale=A, v_scale=A + 2)):
        assert f(_cache(**bad)) == -2, bad
    for far in (dict(k_stride=[8 << 32, 128, 64]), dict(v_stride=[2048, 128, 8 << 32]),
                dict(dtype=1, k_scale=A, v_scale=A, scale_stride=[1 << 32, 1, 1])):
        assert f(_cache(**far)) == -3, far
    ok = _cache()
    assert f(ok, Hq=3) == -1 and f(ok, Hq=0) == -1 and f(ok, B=-1) == -1 and f(ok, window=-1) == -1
    assert f(ok, width=-1) == -1 and f(ok, width=1 << 27) == -1
    assert f(ok, q=None) == -1 and f(ok, lens=None) == -1 and f(ok, out=None) == -1 and f(ok, table=None) == -1
    assert f(ok, ws=None) == -6 and f(ok, n=8) == -6 and f(ok, ws=A + 4) == -2 and f(ok, q=A + 2) == -2
    assert f(ok, B=0, q=None, lens=None, out=None, ws=None) == 0
    size = lib.s3d8_paged_attention_workspace_size
    assert size(ctypes.byref(ok), 1, 4) > 0 and size(ctypes.byref(ok), 0, 4) == 0 and size(ctypes.byref(ok), 1, 3) == 0


@no_device_only
def test_rope_append_rejects(lib):
    two = ctypes.c_int64 * 2

    def f(q=A, k=A, v=A, qs=(256, 64), cos=A, sin=A, mp=8, rot=64, pos=A, T=2, Hq=4, table=A, rows=2, width=2, c=None, o=A):
        return lib.s3d8_rope_append(q, two(*qs), k, two(128, 64), v, two(128, 64), cos, sin, mp, rot, 0, pos, None, T, Hq,
                                    table, rows, width, ctypes.byref(c or _cache()), o, None)

    assert f(rot=3) == -1 and f(rot=66) == -1 and f(rot=-2) == -1 and f(mp=-1) == -1 and f(T=-1) == -1 and f(Hq=0) == -1
    assert f(q=None) == -1 and f(pos=None) == -1 and f(o=None) == -1 and f(cos=None) == -1 and f(table=None) == -1
    assert f(qs=(256, -64)) == -1 and f(qs=(260, 64)) == -2 and f(k=A + 8) == -2 and f(cos=A + 2) == -2
    assert f(c=_cache(dim=40)) == -1
    assert f(T=0, q=None, k=None, v=None, pos=None, o=None) == 0


@no_device_only
def test_page_calls_reject(lib):
    layers = (KVCacheStruct * 2)(_cache(), _cache())
    unlike = (KVCacheStruct * 2)(_cache(), _cache(pages=11))
    big = 1 << 20

    assert lib.s3d8_copy_pages(layers, 0, A, A, 1, None) == -1 and lib.s3d8_copy_pages(None, 1, A, A, 1, None) == -1
    assert lib.s3d8_copy_pages(unlike, 2, A, A, 1, None) == -1 and lib.s3d8_copy_pages(layers, 2, None, A, 1, None) == -1
    assert lib.s3d8_copy_pages(layers, 2, A + 2, A, 1, None) == -2 and lib.s3d8_copy_pages(layers, 2, A, A, -1, None) == -1
    assert lib.s3d8_copy_pages(layers, 2, None, None, 0, None) == 0

    def extend(table=A, rows=4, width=3, lens=A, refs=A, pages=10, page=16, seqs=A, add=A, n=2, got=A, ws=A, size=big):
        return lib.s3d8_extend_pages(table, rows, width, lens, refs, pages, page, seqs, add, n, got, ws, size, None)

    assert extend(table=None) == -1 and extend(refs=None) == -1 and extend(lens=None) == -1 and extend(n=5) == -1
    assert extend(n=-1) == -1 and extend(page=0) == -1 and extend(pages=0) == -1 and extend(seqs=None) == -1
    assert extend(add=None) == -1 and extend(got=None) == -1 and extend(ws=None) == -6 and extend(size=8) == -6
    assert extend(ws=A + 4) == -2 and extend(refs=A + 1) == -2 and extend(n=0, seqs=None, add=None, got=None) == 0

    def fork(l=layers, n=2, refs=A, got=A, size=big):
        return lib.s3d8_fork_pages(l, 2, A, 4, 3, A, refs, A, A, n, got, A, size, None)

    assert fork(l=unlike) == -1 and fork(refs=None) == -1 and fork(got=None) == -1 and fork(n=5) == -1
    assert fork(size=8) == -6 and fork(n=0) == 0

    free = lib.s3d8_free_pages
    assert free(A, 4, 3, A, None, 10, A, 2, None) == -1 and free(A, 4, 3, None, A, 10, A, 2, None) == -1
    assert free(A, 4, 3, A, A, 10, A, 5, None) == -1 and free(A, 4, 3, A, A, 10, None, 0, None) == 0

    def compact(live=A, ws=A, size=big, refs=A):
        return lib.s3d8_compact_pages(layers, 2, A, 4, 3, refs, live, ws, size, None)

    assert compact(live=None) == -1 and compact(refs=None) == -1 and compact(size=8) == -6 and compact(ws=A + 4) == -2
    size = lib.s3d8_pages_workspace_size
    assert size(0, 4) == 0 and size(10, -1) == 0 and size(10, 4) >= (30 + 12) * 4


def test_binding_refuses_cpu_tensors(lib):
    bf = torch.bfloat16
    x = torch.zeros((2, 64), dtype=bf)
    with pytest.raises(ValueError):
        s3d8.residual_norm(x, w_pre=x[0])
    kv = torch.zeros((2, 4, 1, 64), dtype=bf)
    with pytest.raises(ValueError):
        s3d8.KVCache(kv, kv)
    with pytest.raises(ValueError):
        s3d8.KVCache(kv, kv[:1])
    with pytest.raises(TypeError):
        s3d8.KVCache(kv.float(), kv.float())
