"""GPU tests of what is done with the pages of the 4-bit cache: forking and freeing (tables, copies), and
moving accepted tokens, bit for bit against tests/tree_ref.py."""
import random

import numpy as np
import pytest
import torch

import tree_ref as tr

pytestmark = pytest.mark.gpu
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731


class Pool:
    """Layers of random pages, with bytes between the layers that belong to nobody."""

    def __init__(self, layers, pages, heads, D, G, page, seed=0, gap=64):
        self.at = tr.Bytes(heads, D, G, page)
        self.layers, self.pages, self.layout = layers, pages, (heads, D, G, page)
        self.size = heads * (page // 32) * self.at.size
        self.stride = pages * self.size + gap
        self.raw = np.random.default_rng(seed).integers(0, 256, (layers, self.stride), dtype=np.uint8)
        self.dev = torch.from_numpy(self.raw).cuda()

    def layer(self, raw, i):
        return self.at.blocks(raw[i, :self.pages * self.size].reshape(self.pages, self.size))


# ---- fork ------------------------------------------------------------------------------------------
def run_fork(w4, pool, table, lens, parent, keep, room, pinned, stream=None):
    B, R, W = len(table), len(parent), len(table[0])
    out = torch.full((R + 1, W), 77, dtype=torch.int32, device="cuda")
    held = torch.full((R + 1,), 77, dtype=torch.int32, device="cuda")
    missing = torch.full((2,), 77, dtype=torch.int32, device="cuda")
    opt = lambda x: None if x is None else i32(x)  # noqa: E731
    pin = None if pinned is None else torch.tensor(pinned, dtype=torch.uint8, device="cuda")
    w4.w4a16_kv4_fork(pool.dev, i32(table), i32(lens), i32(parent), opt(keep), opt(room), pin, out, held, missing, B, R, pool.layers, pool.stride,
                      *pool.layout, pool.pages, W, stream)
    out, held, missing = out.cpu(), held.cpu(), missing.cpu()
    assert (out[R] == 77).all() and held[R] == 77 and missing[1] == 77
    return out[:R].tolist(), held[:R].tolist(), int(missing[0])


def check_fork(w4, pool, table, lens, parent, keep=None, room=None, pinned=None):
    page = pool.layout[3]
    want = tr.fork(table, lens, parent, keep, room, pinned, pool.pages, page)
    got = run_fork(w4, pool, table, lens, parent, keep, room, pinned)
    assert got[1] == want[1] and got[2] == want[2]
    assert got[0] == want[0]
    expect = pool.raw.copy()
    for i in range(pool.layers):
        blocks = pool.layer(expect, i)
        for src, dst, n in want[3]:
            blocks[dst, :, :-(-n // 32)] = blocks[src, :, :-(-n // 32)]
    assert np.array_equal(pool.dev.cpu().numpy(), expect)
    return want


def random_fork(r, pages, batch, width, page, rows):
    ids = r.sample(range(pages), pages)
    table, lens = [], []
    for _ in range(batch):
        n = r.choice([0, 1, page - 1, page, page + 1, r.randint(0, width * page), r.randint(0, 3 * page)])
        n = min(n, width * page)
        used = -(-n // page)
        row = (ids[:used] + [-1] * width)[:width]
        ids = ids[used:]
        if table and r.random() < 0.4:  # a prefix that the row before has too
            c = min(r.randint(0, used), -(-lens[-1] // page))
            row[:c] = table[-1][:c]
        if r.random() < 0.2 and used:
            row[r.randrange(used)] = r.choice([-1, pages, 2 ** 31 - 1, -2 ** 31])
        table.append(row)
        lens.append(n)
    parent = [r.choice([-1, batch, 2 ** 31 - 1, -2 ** 31]) if r.random() < 0.1 else r.randrange(batch) for _ in range(rows)]
    keep = None if r.random() < 0.3 else [r.choice([2 ** 31 - 1, -4, 0, r.randint(0, width * page)]) if r.random() < 0.6 else 2 ** 30 for _ in range(rows)]
    room = None if r.random() < 0.2 else [r.choice([0, -9, 2 ** 31 - 1]) if r.random() < 0.05 else r.randint(0, width * page) for _ in range(rows)]
    pinned = None if r.random() < 0.4 else [int(r.random() < 0.3) * r.randint(1, 255) for _ in range(pages)]
    return table, lens, parent, keep, room, pinned


@pytest.mark.parametrize("layers,heads,D,G,page", [(1, 1, 64, 64, 32), (2, 3, 128, 64, 64), (3, 1, 128, 32, 96), (2, 2, 64, 32, 32), (1, 2, 128, 128, 64)])
def test_fork(lib, layers, heads, D, G, page):
    for seed in range(12):
        r = random.Random(seed)
        pages, width = r.choice([7, 32, 33, 90]), r.randint(1, 6)
        batch, rows = r.randint(1, 9), r.choice([1, 2, 5, 16, 17, 40])
        pool = Pool(layers, pages, heads, D, G, page, seed)
        check_fork(lib, pool, *random_fork(r, pages, batch, width, page, rows))


def test_fork_many_rows_and_pages(lib):
    for seed, pages, batch, rows, width in ((1, 20000, 300, 1023, 40), (2, 20000, 300, 2048, 9), (3, 1 << 19, 70, 70, 700), (4, 50, 3, 1500, 2)):
        r = random.Random(seed)
        pool = Pool(1, pages, 1, 64, 64, 32, seed)
        table, lens, parent, keep, room, pinned = random_fork(r, pages, batch, width, 32, rows)
        if seed == 3:
            pinned = [1] * (pages - 900) + [0] * 900  # the free ones are the last
        check_fork(lib, pool, table, lens, parent, keep, room, pinned)


def test_fork_of_beams(lib):
    """What is shared, copied and freed, spelled out."""
    pool = Pool(2, 10, 1, 128, 64, 64)
    table = [[3, 5, -1, -1], [3, 8, -1, -1]]          # two beams of 100 tokens that share their first page
    got = check_fork(lib, pool, table, [100, 100], [1, 1, 0, 1], None, [101, 101, 130, 101], None)
    # the first that goes on in page 8 keeps it, as does the one in page 5; the others copy it to the lowest free pages
    assert got[0] == [[3, 8, -1, -1], [3, 0, -1, -1], [3, 5, 1, -1], [3, 2, -1, -1]]
    assert got[2] == 0 and got[3] == [(8, 0, 36), (8, 2, 36)]
    pool = Pool(1, 10, 1, 128, 64, 64)
    # 64 tokens kept whole by one row and 20 of them by another: the second has a copy; page 5 is free again
    got = check_fork(lib, pool, table, [100, 100], [0, 0], [64, 20], None, None)
    assert got[0] == [[3, -1, -1, -1], [0, -1, -1, -1]] and got[3] == [(3, 0, 20)]
    pool = Pool(1, 10, 1, 128, 64, 64)
    got = check_fork(lib, pool, table, [100, 100], [0], [20], [128], [0, 0, 0, 1, 0, 0, 0, 0, 0, 0])  # the page is pinned
    assert got[0] == [[0, 1, -1, -1]] and got[3] == [(3, 0, 20)]
    pool = Pool(1, 4, 1, 128, 64, 64)
    got = check_fork(lib, pool, [[0, 1]], [100], [0, 0, 0], None, [128, 128, 128], None)  # pages for one of two copies... and the other
    assert got[2] == 0 and got[0] == [[0, 1], [0, 2], [0, 3]]
    pool = Pool(1, 3, 1, 128, 64, 64)
    got = check_fork(lib, pool, [[0, 1]], [100], [0, 0, 0], None, None, None)
    assert got[2] == 1 and got[0] == [[0, 1], [0, 2], [0, -1]]


def test_fork_on_a_side_stream_and_in_a_graph(lib):
    r = random.Random(5)
    pool = Pool(2, 64, 2, 64, 64, 32, 5)
    table = i32([[8 * b + i for i in range(6)] + [-1] * 2 for b in range(6)])
    lens, parent = i32([180, 170, 33, 64, 1, 0]), i32([0, 0, 1, 2, 2, 2])
    room = i32([200] * 6)
    out, held, missing = torch.zeros_like(table), torch.zeros_like(lens), i32([9])

    def call(out, held, missing, stream=None):
        lib.w4a16_kv4_fork(pool.dev, table, lens, parent, None, room, None, out, held, missing, 6, 6, 2, pool.stride, *pool.layout, 64, 8, stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(out, held, missing, side)
    for i in range(3):
        parent.copy_(i32([(i + j) % 7 - 1 for j in range(6)]))
        now = torch.zeros_like(table), torch.zeros_like(lens), i32([9])
        call(*now)
        torch.cuda.synchronize()
        after = pool.dev.clone()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(now, (out, held, missing))) and torch.equal(pool.dev, after)


# ---- compact -----------------------------------------------------------------------------------------
def check_compact(w4, pool, spread, table, path, count, max_new=None, stream=None):
    heads, D, G, page = pool.layout
    rows = [0]
    for n, _ in spread:
        rows.append(rows[-1] + n)
    B, most, W = len(spread), len(path[0]), len(table[0])
    out = torch.full((B + 1,), 77, dtype=torch.int32, device="cuda")
    max_new = max_new or max(1, max(n for n, _ in spread))
    w4.w4a16_kv4_compact(pool.dev, i32(path), i32(count), i32(rows), i32([L for _, L in spread]), i32(table), out, B, max(1, rows[-1]), max_new,
                         most, pool.layers, pool.stride, heads, D, G, page, pool.pages, W, stream)
    expect, lens = pool.raw.copy(), []
    for b, (n, L) in enumerate(spread):
        L = max(0, L)
        real = min(n, max_new)
        held = L - n
        k = max(0, min(count[b], most, real))
        lens.append(max(0, held + k))

        def where(pos):
            at = pos // page
            p = table[b][at] if 0 <= pos and at < W else -1
            return (p, pos % page) if 0 <= p < pool.pages else None

        for i in range(pool.layers):
            blocks = pool.layer(expect, i)
            had = {}
            for j in range(k):
                if j < path[b][j] < real and where(held + j) and where(held + path[b][j]):
                    had[j] = pool.at.take(blocks, *where(held + path[b][j]))
            for j, x in had.items():
                pool.at.put(blocks, *where(held + j), *x)
    got = out.cpu().tolist()
    assert got[:B] == lens and got[B] == 77
    assert np.array_equal(pool.dev.cpu().numpy(), expect)
    return out


def tables(r, spread, page, extra=1):
    used = [max(0, -(-L // page)) for _, L in spread]
    pages = sum(used) + 2
    ids, at, W = r.sample(range(pages), pages), 0, max(used + [1]) + extra
    table = []
    for u in used:
        table.append(ids[at:at + u] + [-1] * (W - u))
        at += u
    return pages, table


@pytest.mark.parametrize("layers,heads,D,G,page", [(1, 1, 64, 64, 32), (2, 3, 128, 64, 64), (3, 1, 128, 32, 96), (2, 2, 64, 32, 32), (1, 2, 128, 128, 64)])
def test_compact(lib, layers, heads, D, G, page):
    for seed in range(6):
        r = random.Random(seed)
        spread = [(n, n + r.choice([0, 1, 29, 31, 32, 60, 130])) for n in (1, 0, 40, 26, 7, 64, 9)] + [(5, 3)]
        pages, table = tables(r, spread, page)
        most = r.choice([1, 5, 9, 30])
        path, count = [], []
        for n, _ in spread:
            k = min(most, n)
            p = sorted(r.sample(range(n), r.randint(0, k))) if n else []
            if seed % 2:  # branches that stay partly in place, neighbours that overlap
                p = [i if r.random() < 0.4 else min(n - 1, i + 1) for i in range(k)]
            path.append((p + [r.choice([-1, 0, 2 ** 31 - 1])] * most)[:most])
            count.append(len(p))
        check_compact(lib, Pool(layers, pages, heads, D, G, page, seed), spread, table, path, count)


def test_compact_long_branches_and_odd_arguments(lib):
    r = random.Random(7)
    spread = [(200, 233), (90, 90), (64, 100)]
    pages, table = tables(r, spread, 32)
    path = [sorted(r.sample(range(200), 150)), list(range(1, 90)) + [89] * 61, [min(63, 2 * j) for j in range(150)]]
    check_compact(lib, Pool(2, pages, 2, 128, 64, 32, 1), spread, table, path, [150, 89, 32])
    # counts out of range; entries that do not ascend, that are no node; places and nodes without a page; nodes past the most
    table[0][2], table[1][1], table[2][3] = -1, pages, 2 ** 31 - 1
    path = [[5, 0, 199, 200, -3, 2 ** 31 - 1, 150, 8, 8, 70], [40, 3, 2, 60, 60, 89, 5, 6, 7, 33], [63] * 10]
    check_compact(lib, Pool(1, pages, 1, 64, 32, 32, 2), spread, table, path, [10, 2 ** 31 - 1, -5])
    check_compact(lib, Pool(1, pages, 1, 64, 32, 32, 3), spread, table, path, [10, 10, 10], max_new=61)


def test_compact_many_layers(lib):
    """More units than waves: each wave goes through several."""
    r = random.Random(8)
    spread = [(8, 8 + i % 40) for i in range(60)]
    pages, table = tables(r, spread, 32)
    path = [sorted(r.sample(range(8), 4)) for _ in spread]
    check_compact(lib, Pool(70, pages, 5, 64, 64, 32, 4, gap=0), spread, table, path, [r.randint(0, 4) for _ in spread])


def test_compact_in_a_graph(lib):
    r = random.Random(9)
    spread = [(20, 50), (20, 31)]
    pages, table = tables(r, spread, 32)
    pool = Pool(2, pages, 2, 64, 64, 32, 6)
    path, count, rows, lens, tab = i32([[0, 3, 9, 11], [2, 4, 6, 19]]), i32([4, 3]), i32([0, 20, 40]), i32([50, 31]), i32(table)
    out = torch.zeros_like(lens)

    def call(out, stream=None):
        lib.w4a16_kv4_compact(pool.dev, path, count, rows, lens, tab, out, 2, 40, 20, 4, 2, pool.stride, *pool.layout, pages, len(table[0]), stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(out, side)
    for i in range(3):
        pool.dev.random_(0, 256)
        path.copy_(i32([[0, 3 + i, 9, 11], [2, 4, 6 + i, 19]]))
        before = pool.dev.clone()
        call(torch.zeros_like(out))
        torch.cuda.synchronize()
        want = pool.dev.clone()
        pool.dev.copy_(before)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(pool.dev, want) and out.tolist() == [34, 14]


# ---- past 4 GiB -------------------------------------------------------------------------------------
def test_layers_past_4_gib(lib):
    """Two layers 5 GiB apart, pages in the last of each layer's bytes: the same tokens move, the same page is
    copied as in a small pool."""
    heads, D, G, page = 8, 128, 64, 256
    size = lib.w4a16_kv4_page_bytes(heads, D, G, page)
    pages = (5 << 30) // size
    stride = pages * size
    big = torch.zeros(2 * stride, dtype=torch.uint8, device="cuda").view(2, pages, size)
    ids = [pages - 1, pages - 3, 5]
    small = Pool(2, 3, heads, D, G, page, 1, gap=0)
    big[:, ids] = small.dev.view(2, 3, size)
    spread, path, count = [(40, 270)], [[0, 9, 11, 39]], [4]  # the tree begins in one page and ends in another
    check_compact(lib, small, spread, [[0, 1, -1]], path, count)
    out = i32([0])
    lib.w4a16_kv4_compact(big, i32(path), i32(count), i32([0, 40]), i32([270]), i32([[ids[0], ids[1], -1]]), out, 1, 40, 40, 4, 2, stride, heads, D, G,
                          page, pages, 3)
    assert out.item() == 234 and torch.equal(big[:, ids], small.dev.view(2, 3, size))
    # page `pages - 2` is the only free one
    pinned = torch.ones(pages, dtype=torch.uint8, device="cuda")
    pinned[pages - 2] = 0
    table, held, missing = torch.zeros(1, 2, dtype=torch.int32, device="cuda"), i32([0]), i32([7])
    lib.w4a16_kv4_fork(big, i32([[ids[0], ids[1]]]), i32([300]), i32([0]), None, None, pinned, table, held, missing, 1, 1, 2, stride, heads, D, G, page, pages, 2)
    assert table.tolist() == [[ids[0], pages - 2]] and missing.item() == 0
    blocks = big.view(2, pages, heads, page // 32, -1)
    assert torch.equal(blocks[:, pages - 2, :, :2], blocks[:, ids[1], :, :2]) and (blocks[:, pages - 2, :, 2:] == 0).all()


def test_fork_with_the_most_pages_in_a_graph(lib):
    """2^19 pages need more LDS than a launch has unasked; one call serves a capture as well."""
    heads, D, G, page, pages, W = 1, 64, 64, 32, 1 << 19, 3
    pool = torch.zeros(pages * lib.w4a16_kv4_page_bytes(heads, D, G, page), dtype=torch.uint8, device="cuda")
    pinned = torch.ones(pages, dtype=torch.uint8, device="cuda")
    free = [7, 70000, 300001, pages - 1]
    pinned[free] = 0
    table, lens, parent, room = i32([[3, 9, -1], [3, pages - 2, -1]]), i32([40, 64]), i32([0, 0, 1]), i32([50, 70, 96])
    out, held, missing = torch.zeros(3, W, dtype=torch.int32, device="cuda"), i32([0] * 3), i32([9])

    def call(stream=None):
        lib.w4a16_kv4_fork(pool, table, lens, parent, None, room, pinned, out, held, missing, 2, 3, 1, pool.numel(), heads, D, G, page, pages, W, stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(side)
    # page 9 is pinned, so both rows copy it
    for _ in range(3):
        out.fill_(5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert out.tolist() == [[3, 7, -1], [3, 70000, 300001], [3, pages - 2, pages - 1]] and held.tolist() == [40, 40, 64] and missing.item() == 0
    pinned[9] = 0
    call()
    assert out.tolist() == [[3, 9, -1], [3, 7, 70000], [3, pages - 2, 300001]]
