"""Host-side checks of the vision decoder's calls (no GPU): argument rejection before any
CUDA call, workspace sizes, and the binding's own checks.  Dummy addresses are never
dereferenced; they are passed only on a machine without a CUDA device."""
import ctypes

import pytest
import torch

import s3d8_a8_linear_gb300 as s3d8
from s3d8_a8_linear_gb300 import _build
from s3d8_a8_linear_gb300.decoder import KVCacheStruct

no_device_only = pytest.mark.skipif(torch.cuda.is_available(),
                                    reason="dummy-pointer rejection tests run only without a GPU")

A, B, C, D = 0x10000, 0x20000, 0x30000, 0x40000
BIG = 1 << 40
two = ctypes.c_int64 * 2


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return s3d8.load()


@no_device_only
def test_norm_rope_rejects(lib):
    def f(q=A, qs=(256, 64), Hq=4, k=B, ks=(128, 64), Hk=2, wq=C, wk=C, cos=A, sin=A, mp=8, rot=64, pos=A, T=2, dim=64,
          qo=D, ko=D):
        return lib.s3d8_norm_rope(q, two(*qs), Hq, k, two(*ks), Hk, wq, wk, cos, sin, mp, rot, 0, pos, T, dim, 1e-5, qo, ko,
                                  None)

    for bad in (dict(dim=0), dict(dim=24), dict(dim=272, rot=0), dict(rot=3), dict(rot=66), dict(rot=-2), dict(T=-1),
                dict(Hq=0), dict(Hk=-1), dict(mp=-1), dict(q=None), dict(k=None), dict(cos=None), dict(sin=None),
                dict(qo=None), dict(ko=None), dict(qs=(-8, 64)), dict(Hk=0, k=None, ko=None), dict(T=(1 << 24) + 1)):
        assert f(**bad) == -1, bad
    for bad in (dict(q=A + 8), dict(qs=(260, 64)), dict(ks=(128, 60)), dict(wq=C + 2), dict(wk=C + 8), dict(qo=D + 8),
                dict(ko=D + 2), dict(cos=A + 2), dict(pos=A + 1)):
        assert f(**bad) == -2, bad
    assert f(T=0, q=None, k=None, qo=None, ko=None) == 0

    def b(dq=A, dqs=(256, 64), dk=B, wq=C, wk=C, dqi=D, dki=D, dwq=A, dwk=A, ws=A, n=1 << 30, T=2, q=A, k=B):
        return lib.s3d8_norm_rope_backward(dq, two(*dqs), dk, two(128, 64), q, two(256, 64), 4, k, two(128, 64), 2, wq, wk,
                                           A, A, 8, 64, 0, A, T, 64, 1e-5, dqi, dki, dwq, dwk, ws, n, None)

    for bad in (dict(dq=None), dict(dk=None), dict(dqi=None), dict(dki=None), dict(dwq=None), dict(wq=None), dict(dwk=None),
                dict(wk=None), dict(q=None)):
        assert b(**bad) == -1, bad
    assert b(ws=None) == -6 and b(n=8) == -6 and b(ws=A + 4) == -2 and b(dqs=(4, 64)) == -2 and b(dwq=A + 2) == -2
    size = lib.s3d8_norm_rope_backward_workspace_size
    assert size(0, 4, 2, 64) == 0 and size(5, 0, 2, 64) == 0 and size(5, 4, 2, 40) == 0 and size(5, 4, 0, 64) >= 2 * 64 * 4


@no_device_only
def test_normed_append_rejects(lib):
    c = KVCacheStruct(k=A, v=B, pages=10, page_size=16, heads=2, dim=64, dtype=0)
    c.k_stride[:] = c.v_stride[:] = [2048, 128, 64]

    def f(wq=C, wk=C, q=A, T=2):
        return lib.s3d8_norm_rope_append(q, two(256, 64), B, two(128, 64), B, two(128, 64), A, A, 8, 64, 0, A, None, T, 4, A,
                                         2, 2, wq, wk, 1e-5, ctypes.byref(c), D, None)

    assert f(wq=C + 8) == -2 and f(wk=C + 2) == -2 and f(q=None) == -1 and f(T=-1) == -1 and f(T=0) == 0


@no_device_only
def test_cross_attention_rejects(lib):
    def f(q=A, qs=(256, 64), k=B, ks=(128, 64), v=B, vs=(128, 64), spans=A, T=3, S=5, Hq=4, heads=2, dim=64, out=D, lse=None,
          ws=A, n=BIG):
        return lib.s3d8_cross_attention(q, two(*qs), k, two(*ks), v, two(*vs), spans, T, S, Hq, heads, dim, 0.125, out, lse,
                                        ws, n, None)

    for bad in (dict(T=-1), dict(S=-1), dict(Hq=0), dict(Hq=3), dict(heads=0), dict(dim=0), dict(dim=12), dict(q=None),
                dict(k=None), dict(v=None), dict(out=None), dict(qs=(-8, 64)), dict(vs=(128, -64)), dict(T=(1 << 24) + 1)):
        assert f(**bad) == -1, bad
    for bad in (dict(dim=136), dict(Hq=258), dict(T=1 << 20, Hq=4096, heads=64)):
        assert f(**bad) == -3, bad
    for bad in (dict(q=A + 8), dict(k=B + 2), dict(ks=(132, 64)), dict(vs=(128, 4)), dict(spans=A + 4), dict(out=D + 8),
                dict(lse=A + 2), dict(ws=A + 8)):
        assert f(**bad) == -2, bad
    assert f(ws=None) == -6
    assert f(T=0, q=None, out=None, ws=None) == 0

    def b(dout=A, ds=(256, 64), out=A, lse=A, dq=D, dk=D, dv=D, ws=A, n=BIG, T=3, S=5):
        return lib.s3d8_cross_attention_backward(dout, two(*ds), A, two(256, 64), B, two(128, 64), B, two(128, 64), out, lse,
                                                 A, T, S, 4, 2, 64, 0.125, dq, dk, dv, ws, n, None)

    for bad in (dict(dout=None), dict(out=None), dict(lse=None), dict(dq=None), dict(dk=None), dict(dv=None),
                dict(ds=(256, -8))):
        assert b(**bad) == -1, bad
    for bad in (dict(dout=A + 8), dict(ds=(4, 64)), dict(out=A + 2), dict(lse=A + 1), dict(dq=D + 8), dict(dk=D + 8),
                dict(dv=D + 4), dict(ws=A + 8)):
        assert b(**bad) == -2, bad
    assert b(ws=None) == -6 and b(n=4) == -6 and b(T=0, S=0) == 0
    for size in (lib.s3d8_cross_attention_workspace_size, lib.s3d8_cross_attention_backward_workspace_size):
        assert size(0, 5, 4, 2, 64) == 0 and size(3, 5, 3, 2, 64) == 0 and size(3, 5, 4, 2, 136) == 0
        assert size(3, 5, 4, 2, 64) > 0 and size(3, 0, 4, 2, 64) > 0


@no_device_only
def test_sample_rejects(lib):
    def f(x=A, stride=100, rows=2, V=100, u=A, t=A, k=A, p=A, m=A, out=A, lp=A):
        return lib.s3d8_sample(x, stride, rows, V, u, t, k, p, m, out, lp, None)

    for bad in (dict(x=None), dict(u=None), dict(out=None), dict(rows=-1), dict(V=0), dict(stride=-1)):
        assert f(**bad) == -1, bad
    for bad in (dict(x=A + 1), dict(u=A + 2), dict(t=A + 1), dict(k=A + 2), dict(p=A + 3), dict(m=A + 1), dict(out=A + 2),
                dict(lp=A + 2)):
        assert f(**bad) == -2, bad
    assert f(V=524225, stride=524288) == -3 and f(rows=0, x=None, u=None, out=None) == 0


def test_binding_refuses_before_any_call(lib):
    bf = torch.bfloat16
    x = torch.zeros((2, 4, 64), dtype=bf)
    w = torch.ones(64, dtype=bf)
    for call in (lambda: s3d8.norm_rope(x), lambda: s3d8.norm_rope(x[0]), lambda: s3d8.norm_rope(x, k_norm=w),
                 lambda: s3d8.norm_rope(x, cos=torch.zeros(4, 32)), lambda: s3d8.cross_attention(x, x, x),
                 lambda: s3d8.cross_attention(x, x, x[:1]), lambda: s3d8.cross_attention(x[0], x, x),
                 lambda: s3d8.sample(x[0], torch.zeros(4)), lambda: s3d8.sample(x, torch.zeros(4)),
                 lambda: s3d8.cross_attention_backward(x, x, x, x, x, torch.zeros(2, 4))):
        with pytest.raises((ValueError, TypeError)):
            call()
