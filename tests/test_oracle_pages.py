"""The page operators' oracle against worked examples and against what the
operators have to keep (every row's contents, one reference per holder)."""
import numpy as np
import pytest

from oracle import pages as op


def _i(*x):
    return np.array(x, np.int32)


def _contents(pool, table, held, ctx, r):
    ps = pool.shape[2]
    return np.concatenate([pool[:, table[r, j], :min(ps, int(ctx[r]) - j * ps)]
                           for j in range(-(-int(ctx[r]) // ps))], 1) if ctx[r] else pool[:, :0].reshape(len(pool), 0)


def test_resize_worked_example():
    # pages of 4; row 0 shrinks 3 -> 1, row 1 grows 1 -> 3, row 2 is left alone
    table = _i([5, 2, 0, -1], [1, -1, -1, -1], [4, -1, -1, -1])
    held, refs = _i(3, 1, 1), _i(1, 1, 1, 0, 1, 2, 0)
    t, h, r, st = op.oracle_resize_pages(table, held, refs, _i(4, 9, -1), 4)
    assert st == 0 and h.tolist() == [1, 3, 1]
    assert t.tolist() == [[5, -1, -1, -1], [1, 0, 2, -1], [4, -1, -1, -1]]
    assert r.tolist() == [1, 1, 1, 0, 1, 2, 0]


def test_resize_overflow_keeps_the_row_and_the_growing_rows_behind_it():
    table = np.full((3, 3), -1, np.int32)
    held, refs = _i(0, 0, 0), _i(0, 0, 0)
    t, h, r, st = op.oracle_resize_pages(table, held, refs, _i(2, 3, 1), 1)
    assert st == op.OVERFLOW and h.tolist() == [2, 0, 0] and r.tolist() == [1, 1, 0]
    assert t[0].tolist() == [0, 1, -1] and (t[1:] == -1).all()


def test_fork_worked_example():
    pool = np.arange(6 * 2, dtype=np.int32).reshape(1, 6, 2)
    table = _i([3, 1, -1], [-1, -1, -1], [-1, -1, -1])
    k, v, t, h, r, c, st = op.oracle_fork_pages(pool, pool + 100, table, _i(2, 0, 0), _i(0, 1, 0, 1, 0, 0),
                                                _i(3, 0, 0), _i(0, 0), _i(2, 1))
    assert st == 0 and h.tolist() == [2, 2, 2] and c.tolist() == [3, 3, 3]
    assert t.tolist() == [[3, 1, -1], [3, 2, -1], [3, 0, -1]] and r.tolist() == [1, 1, 1, 3, 0, 0]
    assert k[0, 0, 0] == pool[0, 1, 0] and k[0, 0, 1] == pool[0, 0, 1]      # one used position
    assert v[0, 2, 0] == pool[0, 1, 0] + 100


def test_fork_of_a_row_that_names_a_free_page():
    # pages of 2; the parent names the free pages 0 (full) and 2 (its last, half used)
    pool = np.arange(5 * 2, dtype=np.int32).reshape(1, 5, 2)
    table = _i([1, 0, 2], [-1, -1, -1])
    k, _, t, h, r, c, st = op.oracle_fork_pages(pool, pool, table, _i(3, 0), _i(0, 1, 0, 0, 1), _i(5, 0), _i(0), _i(1))
    assert st == op.BAD_INDEX and h.tolist() == [3, 3] and c.tolist() == [5, 5]
    assert t[1].tolist() == [1, 0, 0] and r.tolist() == [1, 2, 0, 0, 1]      # page 0 is handed out, not shared
    assert (k == pool).all()


def test_copy_skips_pairs_that_depend_on_one_another():
    pool = np.arange(8, dtype=np.int32).reshape(1, 8, 1)
    # 0 -> 1 and 1 -> 2 (reads what the first writes); 3 -> 4 twice; swap 5, 6
    k, _, st = op.oracle_copy_pages(pool, pool, _i(0, 1, 3, 7, 5, 6, -1, 2), _i(1, 2, 4, 4, 6, 5, 0, 2))
    assert st == op.BAD_INDEX
    assert k[0, :, 0].tolist() == [0, 0, 2, 3, 3, 5, 6, 7]


def test_compact_worked_example():
    pool = np.arange(6, dtype=np.int32).reshape(1, 6, 1)
    table = _i([5, 1], [3, -1])
    k, v, t, r, remap, n, st = op.oracle_compact_pages(pool, pool, table, _i(2, 1), _i(0, 1, 0, 2, 0, 1))
    assert n == 3 and st == 0 and t.tolist() == [[2, 1], [0, -1]] and r.tolist() == [2, 1, 1, 0, 0, 0]
    assert remap.tolist() == [-1, 1, -1, 0, -1, 2] and k[0, :3, 0].tolist() == [3, 1, 5]


@pytest.mark.parametrize("seed", range(6))
def test_a_run_of_steps_keeps_every_rows_contents(seed):
    rng = np.random.default_rng(seed)
    R, N, ps, width = 7, 60, 4, 12
    pool = rng.integers(0, 1 << 30, (2, N, ps)).astype(np.int32)
    table, held, refs, ctx = (np.full((R, width), -1, np.int32), np.zeros(R, np.int32),
                              np.zeros(N, np.int32), np.zeros(R, np.int32))
    for _ in range(20):
        new = np.where(rng.random(R) < 0.3, 0, np.minimum(ctx + rng.integers(0, 6, R), width * ps)).astype(np.int32)
        table, held, refs, st = op.oracle_resize_pages(table, held, refs, new, ps)
        ctx = np.minimum(new, held * ps).astype(np.int32)
        empty, full = np.flatnonzero(held == 0), np.flatnonzero(ctx > 0)
        if len(empty) and len(full):
            par, kid = _i(int(full[0])), _i(int(empty[0]))
            was = _contents(pool, table, held, ctx, par[0])
            pool, _, table, held, refs, ctx, st = op.oracle_fork_pages(pool, pool, table, held, refs, ctx, par, kid)
            if st == 0:
                np.testing.assert_array_equal(_contents(pool, table, held, ctx, kid[0]), was)
        before = [_contents(pool, table, held, ctx, r) for r in range(R)]
        pool, _, table, refs, _, n, st = op.oracle_compact_pages(pool, pool, table, held, refs)
        assert st == 0 and (refs[:n] > 0).all() and (refs[n:] == 0).all()
        for r in range(R):
            np.testing.assert_array_equal(_contents(pool, table, held, ctx, r), before[r])
        count = np.zeros(N, np.int64)
        for r in range(R):
            np.add.at(count, table[r, :held[r]], 1)
        np.testing.assert_array_equal(count, refs)
