"""The page calls where entries are many, sums large or page ids wrong, against the
whole-number model of their definitions."""
import numpy as np
import pytest
import torch

import s3d8_a8_linear_gb300 as s3d8
from gpu_util import dev
from test_gpu_kv_cache import Plain, _i32, _lib, _parts, _pool, _same, _state  # noqa: F401

pytestmark = pytest.mark.gpu


def test_forks_of_many_entries_and_wide_rows():
    """Several entries a warp, rows of several columns a lane, some with pages and some without."""
    rng = np.random.default_rng(1)
    pages, rows, width, page, n = 9000, 400, 75, 4, 200
    pool = _pool(1, pages, page, 1, 16, False, "head", 2)
    plain = Plain(np.full((rows, width), -1, np.int32), np.zeros(rows, np.int32), np.zeros(pages, np.int32), page)
    plain.extend(np.arange(n), rng.integers(0, 40 * page, n))
    start = _state(plain)
    before = [t.clone() for t in _parts(pool)]
    parents, children = rng.integers(0, n, n), n + rng.permutation(n)
    expect, copies = plain.fork(parents, children)
    for _ in range(5):
        table, lens, refs = (t.clone() for t in start)
        got = s3d8.fork_pages(pool, table, lens, refs, _i32(parents), _i32(children))
        assert got.tolist() == expect
        _same(plain, table, lens, refs)
        for have, old in zip(_parts(pool), before):
            want = old.clone()
            for a, b, tokens in copies:
                want[b, :tokens] = old[a, :tokens]
            assert torch.equal(have, want)
            have.copy_(old)
