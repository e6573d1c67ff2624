"""The append's ring of bulk copies at layouts where its shared memory is nearly all that a
CTA may have, against the formula in 64 bits."""
import pytest

import test_gpu_kv_cache as kv
from test_gpu_kv_cache import _lib  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("T,heads,group,dim,rotary,interleaved", [
    (400, 32, 1, 96, 96, False), (305, 8, 10, 96, 96, True), (700, 8, 12, 128, 0, False), (400, 29, 1, 80, 80, False),
    (400, 4, 16, 192, 192, False), (333, 8, 9, 128, 64, True), (400, 31, 2, 112, 112, False),
])
def test_append_of_many_heads(T, heads, group, dim, rotary, interleaved, int8):
    kv.test_append_many_tokens(T, heads, group, dim, rotary, interleaved, False, int8)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("T,group,dim,rotary,interleaved", [
    (305, 32, 128, 128, False), (1100, 8, 256, 64, True), (5003, 1, 16, 16, False), (640, 71, 64, 64, False),
    (400, 4, 80, 0, False), (3001, 1, 128, 128, True),
])
def test_append_many_tokens_of_one_key_value_head(T, group, dim, rotary, interleaved, int8):
    """One key/value head (and one query head): the stride of an axis of one element is whatever it is."""
    kv.test_append_many_tokens(T, 1, group, dim, rotary, interleaved, False, int8)
