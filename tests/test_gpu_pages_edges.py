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


@pytest.mark.parametrize("bad", [8, -1, -7, 2 ** 31 - 1])
def test_forks_of_rows_with_pages_out_of_range_are_refused(bad):
    """A wrong page id among the full pages, in the last full one or in the partial one: the
    entry gets 0, an empty child and no page; those behind it take the lowest free ids."""
    pages, page, n = 20, 4, 5
    pool = _pool(2, pages, page, 1, 16, False, "head", 3)
    bad = pages if bad == 8 else bad
    table = np.full((2 * n, 70), -1, np.int32)
    table[0, :3], table[1, :3], table[2, :3], table[3, :3], table[4, :2] = [0, 1, 2], [3, 4, 5], [6, 7, 8], [9, 10, 11], [12, 13]
    plain = Plain(table, np.array([10, 10, 10, 10, 8] + [0] * n, np.int32), np.array([1] * 14 + [0] * 6, np.int32), page)
    for row, col in ((0, 0), (1, 1), (2, 2), (4, 1)):
        plain.table[row, col] = bad
    state = _state(plain)
    before = [t.clone() for t in _parts(pool)]
    assert s3d8.device_status() == 0
    got = s3d8.fork_pages(pool, *state, _i32([0, 1, 2, 3, 4]), _i32([9, 8, 7, 6, 5]))
    assert got.tolist() == [0, 0, 0, 1, 0]
    assert s3d8.device_status() == -7 and s3d8.device_status() == 0
    expect, copies = plain.fork([3], [6])
    assert expect == [1] and copies == [(11, 14, 2)]
    _same(plain, *state)
    for have, want in zip(_parts(pool), before):
        want[14, :2] = want[11, :2]
        assert torch.equal(have, want)


def test_fork_of_a_row_with_a_wrong_page_far_out():
    """The wrong id in a column that only a later round of the lanes reads; behind the row's tokens it does not matter."""
    pool = _pool(1, 300, 2, 1, 16, False, "head", 4)
    plain = Plain(np.full((4, 260), -1, np.int32), np.zeros(4, np.int32), np.zeros(300, np.int32), 2)
    plain.extend([0], [2 * 250])
    plain.table[0, 251] = 9999
    state = _state(plain)
    assert s3d8.fork_pages(pool, *state, _i32([0]), _i32([1])).tolist() == [1] == plain.fork([0], [1])[0]
    _same(plain, *state)
    assert s3d8.device_status() == 0
    plain.table[0, 231] = state[0][0, 231] = -3
    assert s3d8.fork_pages(pool, *state, _i32([0]), _i32([2])).tolist() == [0]
    assert s3d8.device_status() == -7
    _same(plain, *state)
