"""Caches whose tensors are the same in memory and differ in how torch describes them."""
import pytest
import torch

import s3d8_a8_linear_gb300 as s3d8
from gpu_util import dev
from test_gpu_kv_cache import BF, _i32, _lib, _rand  # noqa: F401

pytestmark = pytest.mark.gpu


def _int8_cache(pages, page, heads, dim, one):
    """`one`: the value scales' axis of one element gets another stride."""
    k, v = (torch.zeros((pages, page, heads, dim), dtype=torch.int8, device=dev()) for _ in "kv")
    ks, vs = (torch.zeros((pages, page, heads), device=dev()) for _ in "kv")
    if one is not None:
        stride = list(vs.stride())
        stride[one] = 977
        vs = vs.as_strided(vs.shape, stride)
    return s3d8.KVCache(k, v, ks, vs)


@pytest.mark.parametrize("pages,page,heads,one", [(6, 16, 1, 2), (9, 1, 3, 1), (1, 64, 2, 0)])
def test_scales_with_any_stride_of_an_axis_of_one(pages, page, heads, one):
    g = torch.Generator().manual_seed(pages)
    T = min(pages * page, 40)
    table, none = _i32([list(range(pages))]), torch.empty((64, 0), device=dev())
    q, k, v = _rand(g, T, 4 * heads, 64), _rand(g, T, heads, 64), _rand(g, T, heads, 64)
    got = []
    for axis in (None, one):
        cache = _int8_cache(pages, page, heads, 64, axis)
        s3d8.rope_append(q, k, v, none, none, _i32(range(T)), cache, table, rows=_i32([0] * T))
        got.append((cache.v_scale.clone(), s3d8.paged_attention(q[:1].contiguous(), cache, table, _i32([T]))))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_scales_laid_out_unlike_are_refused():
    k, v = (torch.zeros((4, 16, 2, 64), dtype=torch.int8, device=dev()) for _ in "kv")
    ks = torch.zeros((4, 16, 2), device=dev())
    with pytest.raises(ValueError):
        s3d8.KVCache(k, v, ks, torch.zeros((4, 2, 16), device=dev()).transpose(1, 2))
    with pytest.raises(ValueError):
        s3d8.KVCache(k, v, ks, ks[:3])
    with pytest.raises(TypeError):
        s3d8.KVCache(k, v, ks, ks.double())
