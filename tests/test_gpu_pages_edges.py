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


def test_growth_that_wants_more_pages_than_an_int_counts():
    """Two entries that want 2^30 pages each between two that want a few, on a table of 2^32 entries."""
    width, pages = 1 << 30, 64
    table = torch.empty((4, width), dtype=torch.int32, device=dev())
    table[:, :8] = -1
    table[:, -8:] = -1
    lens, refs = torch.zeros(4, dtype=torch.int32, device=dev()), torch.zeros(pages, dtype=torch.int32, device=dev())
    space = torch.full((4 * (3 * pages + 3 * 4 + 4),), 255, dtype=torch.uint8, device=dev())
    got = s3d8.extend_pages(table, lens, refs, _i32([2, 0, 3, 1]), _i32([3, width, width, 5]), 1, workspace=space)
    assert got.tolist() == [1, 0, 0, 0]
    assert lens.tolist() == [0, 0, 3, 0] and refs.tolist() == [1] * 3 + [0] * (pages - 3)
    assert table[:, :8].tolist() == [[-1] * 8, [-1] * 8, [0, 1, 2] + [-1] * 5, [-1] * 8]
    assert bool((table[:, -8:] == -1).all())
