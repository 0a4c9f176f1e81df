"""GPU tests of w4a16_kv4_fork where pages run short, and of calls made again after that: what the rows of the
short call keep of the old ones is as it was, bit for bit (layout and definition: tests/tree_ref.py)."""
import random

import numpy as np
import pytest

from test_gpu_pages import Pool, random_fork, run_fork
import tree_ref as tr

pytestmark = pytest.mark.gpu


def again(lib, pool, table, lens, parent, keep, room, pinned):
    """A fork on a pool that an earlier call may have written to: the table of one that never ran short, and
    each row's kept tokens with the bytes that its old row had at the beginning (pool.raw)."""
    page = pool.layout[3]
    want = tr.fork(table, lens, parent, keep, room, pinned, pool.pages, page)
    got = run_fork(lib, pool, table, lens, parent, keep, room, pinned)
    assert got == want[:3]
    raw = pool.dev.cpu().numpy()
    for i in range(pool.layers):
        now, old = pool.layer(raw, i), pool.layer(pool.raw, i)
        for r, p in enumerate(parent):
            for at in range(-(-got[1][r] // page)):
                src, dst, n = table[p][at], got[0][r][at], min(page, got[1][r] - at * page)
                if dst >= 0 and 0 <= src < pool.pages:
                    assert np.array_equal(now[dst, :, :-(-n // 32)], old[src, :, :-(-n // 32)]), (r, at)
    return got


def test_what_a_short_call_leaves(lib):
    """Three pages of 64 tokens: A has 100 tokens in pages 0 and 1, B 40 in page 2."""
    table, lens = [[0, 1], [2, -1]], [100, 40]
    fresh = lambda seed: Pool(2, 3, 1, 128, 64, 64, seed)  # noqa: E731
    # B is not among the rows: its page is free, and is one of the two that the copies of page 1 need
    pool = fresh(1)
    got = run_fork(lib, pool, table, lens, [0, 0, 0], None, None, None)
    assert got == ([[0, 1], [0, 2], [0, -1]], [100] * 3, 1)
    raw = pool.dev.cpu().numpy()
    for i in range(2):
        now, old = pool.layer(raw, i), pool.layer(pool.raw, i)
        assert np.array_equal(now[:2], old[:2]) and np.array_equal(now[2, :, :2], old[1, :, :2])
    got = again(lib, pool, table, lens, [0, 0], None, None, None)
    assert got == ([[0, 1], [0, 2]], [100] * 2, 0)
    # pinned, or kept by a row, B outlives the call that runs short
    pool = fresh(2)
    assert run_fork(lib, pool, table, lens, [0, 0, 0], None, None, [0, 0, 1])[2] == 2
    assert np.array_equal(pool.dev.cpu().numpy(), pool.raw)
    assert again(lib, pool, table, lens, [0, 1], None, None, None)[0] == [[0, 1], [2, -1]]
    pool = fresh(3)
    assert run_fork(lib, pool, table, lens, [0, 0, 1], None, None, None)[2] == 1
    assert again(lib, pool, table, lens, [1, 0], [30, 100], [30, 128], None)[0] == [[2, -1], [0, 1]]


@pytest.mark.parametrize("page", [32, 96])
def test_fewer_rows_after_a_short_call(lib, page):
    short = 0
    for seed in range(40):
        r = random.Random(seed)
        pages, width, batch, rows = r.choice([7, 33]), r.randint(1, 6), r.randint(1, 9), r.choice([5, 16, 40])
        pool = Pool(2, pages, 2, 64, 64, page, seed)
        table, lens, parent, keep, room, pinned = random_fork(r, pages, batch, width, page, rows)
        parent = [p if 0 <= p < batch // 2 + 1 else -1 for p in parent]  # the other old rows are dropped
        if run_fork(lib, pool, table, lens, parent, keep, room, pinned)[2] == 0:
            continue
        short += 1
        some = sorted(r.sample(range(rows), r.randint(1, rows // 2)))
        keep = [keep[i] if keep else 2 ** 30 for i in some]
        keep = [k if r.random() < 0.5 else min(k, r.randint(0, width * page)) for k in keep]
        again(lib, pool, table, lens, [parent[i] for i in some], keep, None, pinned)
    assert short >= 5
