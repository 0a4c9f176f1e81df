"""GPU tests of w4a16_kv4_fork where a wave copies for several rows: from layers * kv_heads * rows = 32768 on, up to
64 rows a wave.  Every byte, as tests/test_gpu_pages.py compares them."""
import random

import pytest

from test_gpu_pages import Pool, check_fork

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layers,heads,rows", [
    (70, 8, 200),     # 6 rows a wave, 2 in the last group
    (70, 8, 59),      # 2 rows a wave, one in the last group
    (560, 8, 259)])   # 64 rows a wave (70 if there were no limit), 3 in the last group
def test_copies_of_several_rows_by_one_wave(lib, layers, heads, rows):
    r = random.Random(rows)
    page, width, batch = 32, 3, 23
    used = [r.choice([1, 2, 3]) for _ in range(batch)]
    pages = sum(used) + rows + 5
    ids, at, table, lens = r.sample(range(pages), sum(used)), 0, [], []
    for u in used:
        table.append(ids[at:at + u] + [-1] * (width - u))
        lens.append(page * u - r.choice([0, 1, 9, 31]))
        at += u
    parent = [r.choice([-1, r.randrange(batch), r.randrange(batch), 3]) for _ in range(rows)]
    keep = [r.choice([2 ** 30, r.randint(0, page * width)]) for _ in range(rows)]
    room = [r.randint(0, page * width) for _ in range(rows)]
    pinned = [int(r.random() < 0.05) for _ in range(pages)]
    table[5][0] = -1                          # an old row without its first page
    pool = Pool(layers, pages, heads, 64, 64, page, rows)
    got = check_fork(lib, pool, table, lens, parent, keep, room, pinned)
    assert len(got[3]) > rows // 4            # copies in most groups, several in each
