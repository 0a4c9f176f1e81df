"""GPU tests of drafted trees over the 4-bit cache: masks and positions, and attention by them, against
tests/tree_ref.py."""
import math
import random

import numpy as np
import pytest
import torch

import decoder_ref as ref
import tree_ref as tr

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731


# ---- masks -------------------------------------------------------------------------------------
def run_tree(w4, parents, lens, window=0, words=None, max_new=None, pad=0, stream=None):
    rows = [0]
    for p in parents:
        rows.append(rows[-1] + len(p))
    flat = [x for p in parents for x in p] + [9] * pad
    n = len(flat)
    max_new = max_new or max(1, max(len(p) for p in parents))
    words = words or (max_new + 31) // 32
    mask = torch.full((n, words), 77, dtype=torch.int32, device="cuda")
    depth, pos = (torch.full((n,), 77, dtype=torch.int32, device="cuda") for _ in range(2))
    w4.w4a16_kv4_tree(i32(flat), i32(rows), i32(lens), mask, depth, pos, len(parents), n, max_new, words, window, stream)
    return mask.cpu(), depth.cpu(), pos.cpu(), rows


@pytest.mark.parametrize("window", [0, 1, 3, 40])
@pytest.mark.parametrize("kind", ["chain", "star", "forest", "tree"])
def test_masks(lib, kind, window):
    r = random.Random(window)
    sizes = [1, 0, 31, 32, 33, 64, 65, 250, 1]
    parents = [tr.trees(r, kind, n) for n in sizes]
    lens = [n + r.choice([0, 5, 1000]) for n in sizes]
    for words in (8, 11):
        mask, depth, pos, rows = run_tree(lib, parents, lens, window, words, pad=2)
        for b, p in enumerate(parents):
            lines = tr.branches(p)
            mine = slice(rows[b], rows[b + 1])
            assert np.array_equal(mask[mine].numpy().view(np.uint32), tr.mask_rows(lines, words, window))
            d = [len(x) - 1 for x in lines]
            assert depth[mine].tolist() == d and pos[mine].tolist() == [lens[b] - len(p) + x for x in d]
        assert (mask[-2:] == 77).all() and (depth[-2:] == 77).all() and (pos[-2:] == 77).all()


def test_masks_of_the_largest_tree_and_bad_parents(lib):
    n = 4096
    chain = [i - 1 for i in range(n)]
    odd = [i if i % 3 == 0 else i + 7 if i % 3 == 1 else i - 1 for i in range(n)]  # a parent must lie before its node
    far = [2 ** 31 - 1, -2 ** 31] + [i - 2 for i in range(2, n)]
    mask, depth, pos, rows = run_tree(lib, [chain, odd, far], [n, n + 3, 5000])
    for b, p in enumerate((chain, odd, far)):
        lines = tr.branches(p)
        assert np.array_equal(mask[rows[b]:rows[b + 1]].numpy().view(np.uint32), tr.mask_rows(lines, 128))
        assert depth[rows[b]:rows[b + 1]].tolist() == [len(x) - 1 for x in lines]


def test_masks_of_nodes_past_the_most_are_left_alone(lib):
    mask, depth, pos, rows = run_tree(lib, [[-1, 0, 1, 1, 2], [-1, 0]], [105, 2], max_new=3)
    assert depth.tolist() == [0, 1, 2, 77, 77, 0, 1] and pos.tolist() == [100, 101, 102, 77, 77, 0, 1]
    assert mask[:, 0].tolist() == [1, 3, 7, 77, 77, 1, 3]


# ---- attention ------------------------------------------------------------------------------------
class Trees:
    """Random pages that hold the tokens before the trees and the nodes, and what is asked of them."""

    def __init__(self, spread, heads, ratio, D, G, page, t, kind="tree", seed=0, extra_words=0, pad_rows=0):
        g, r = np.random.default_rng(seed), random.Random(seed)
        self.spread, self.heads, self.ratio, self.D, self.G, self.page, self.t = spread, heads, ratio, D, G, page, t
        self.at = tr.Bytes(heads, D, G, page)
        used = [max(0, -(-L // page)) for _, L in spread]
        self.pages, self.width = sum(used) + 2, max(used + [1]) + 1
        order = g.permutation(self.pages)
        self.table = np.full((len(spread), self.width), -1, np.int32)
        n = 0
        for b, u in enumerate(used):
            self.table[b, :u] = order[n:n + u]
            n += u
        self.rows = np.concatenate([[0], np.cumsum([n for n, _ in spread])]).astype(np.int32)
        self.lens = np.array([L for _, L in spread], np.int32)
        self.tokens = max(1, int(self.rows[-1])) + pad_rows
        self.max_new, self.max_len = max([n for n, _ in spread] + [1]), max([L for _, L in spread] + [1])
        self.words = (self.max_new + 31) // 32 + extra_words
        self.raw = g.integers(0, 256, (self.pages, heads * (page // 32) * self.at.size), dtype=np.uint8)
        half = self.at.blocks(self.raw)[..., 32 * D:].view(np.float16).reshape(self.pages, heads, page // 32, 2 * D // G, 2, 32)
        half[..., 0, :] = g.uniform(0.02, 0.4, half[..., 0, :].shape)
        half[..., 1, :] = -7.5 * half[..., 0, :].astype(np.float32) + g.standard_normal(half[..., 1, :].shape) * 0.4
        self.parents = [tr.trees(r, kind, n) for n, _ in spread]
        self.lines = [tr.branches(p) for p in self.parents]
        self.mask = np.zeros((self.tokens, self.words), np.uint32)
        self.depth = np.zeros(self.tokens, np.int32)
        self.q = torch.from_numpy(g.standard_normal((self.tokens, heads * ratio * D + 8)).astype(np.float32)).to(t)
        self.g, self.window = g, 0

    def masks(self, window=0):
        self.window = window
        for b, lines in enumerate(self.lines):
            self.mask[self.rows[b]:self.rows[b + 1]] = tr.mask_rows(lines, self.words, window)
            self.depth[self.rows[b]:self.rows[b + 1]] = [len(x) - 1 for x in lines]

    def run(self, w4, max_len=None, scale=None, stream=None, out=None, lse=None, q=None, raw=None):
        w = self.heads * self.ratio * self.D
        if out is None:
            out = torch.full((self.tokens, w + 16), math.nan, dtype=self.t, device="cuda")
            lse = torch.full((self.tokens, self.heads * self.ratio), math.nan, device="cuda")
        self.dev = [torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in (self.rows, self.lens, self.table, self.raw, self.mask.view(np.int32), self.depth)]
        rows, lens, table, raw, mask, depth = self.dev
        self.call = lambda out, lse, q, stream: w4.w4a16_kv4_tree_attention(
            q, rows, lens, table, raw, mask, depth if self.window else None, out, lse, len(self.spread), self.tokens, self.max_new,
            max_len or self.max_len, self.words, w + 8, w + 16, self.heads * self.ratio, self.heads, self.D, self.G, self.page, self.pages, self.width,
            self.window, scale or self.D ** -0.5, w4.DT_BF16 if self.t == BF16 else w4.DT_F16, stream)
        self.call(out, lse, self.q.cuda() if q is None else q, stream)
        return out, lse

    def is_wide(self, w4, max_len=None):
        got = w4.w4a16_kv4_tree_workspace_bytes(len(self.spread), self.tokens, self.max_new, max_len or self.max_len,
                                                self.heads * self.ratio, self.heads, self.D, self.window)
        return got > 4 * (512 + 1024 * 16 * (self.D + 2))  # more than narrow tiles can need

    def seen(self, b):
        n, L = self.spread[b]
        L = max(0, L)
        held = self.spread[b][1] - n
        pos = np.arange(L)
        page = np.where(pos // self.page < self.width, self.table[b][np.minimum(pos // self.page, self.width - 1)], -1)
        have = (page >= 0) & (page < self.pages)
        out = np.zeros((n, L), bool)
        for i in range(n):
            row = self.rows[b] + i
            d = min(max(int(self.depth[row]), 0), n - 1)
            out[i] = (pos < held) & ((pos > held + d - self.window) if self.window else True)
            for j in range(min(n, 32 * self.words)):
                if held + j >= 0 and self.mask[row, j // 32] >> (j % 32) & 1:
                    out[i, held + j] = True
        return torch.from_numpy(out & have), np.where(have, page, 0), pos % self.page

    def check(self, out, lse, scale=None):
        scale = scale or self.D ** -0.5
        out, lse = out.cpu(), lse.cpu().double()
        w, step = self.heads * self.ratio * self.D, ref.half_step(self.t)
        assert out[:, w:].isnan().all()
        assert out[self.rows[-1]:].isnan().all() and lse[self.rows[-1]:].isnan().all()
        vals = self.at.values(self.raw)
        for b, (n, L) in enumerate(self.spread):
            if n == 0:
                continue
            seen, page, place = self.seen(b)
            mine = slice(self.rows[b], self.rows[b + 1])
            for h in range(self.heads * self.ratio):
                k, v = (torch.from_numpy(vals[i, page, h // self.ratio, place]) for i in (0, 1))
                o, l, otol, ltol = tr.attend(self.q[mine, h * self.D:(h + 1) * self.D].double(), k, v, seen, scale)
                got = out[mine, h * self.D:(h + 1) * self.D].double()
                # a query with an infinity has the result NaN by the formula, and its row alone has
                bad = o.isnan().any(1)
                assert torch.equal(got.isnan().any(1), bad) and torch.equal(lse[mine, h].isnan(), bad), (b, h)
                off = (got - o).abs()
                assert (off <= step * o.abs() + otol * (1 + step) + 2.0 ** -25)[~bad].all(), (b, h, float((off - otol)[~bad].max()))
                got = lse[mine, h][~bad]
                l, ltol = l[~bad], ltol[~bad]
                none = l == -math.inf
                assert torch.equal(got == -math.inf, none), (b, h)
                assert ((got - l).abs()[~none] <= ltol[~none]).all(), (b, h)


NARROW = [(26, 26), (1, 1), (5, 300), (33, 70), (0, 40), (2, 64), (64, 97), (9, 9 + 31), (3, 700)]
WIDE = [(40, 40), (17, 330), (0, 3), (129, 300), (64, 96), (33, 45), (1, 65), (100, 140)]


@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("D,G,heads,ratio,page,window,kind", [
    (128, 128, 2, 1, 64, 0, "tree"), (128, 64, 1, 4, 32, 0, "chain"), (128, 32, 1, 2, 96, 0, "forest"), (64, 64, 2, 3, 64, 0, "star"),
    (64, 32, 1, 8, 32, 0, "tree"), (128, 64, 1, 2, 64, 20, "tree"), (64, 32, 2, 1, 32, 1, "chain"), (128, 128, 1, 3, 32, 70, "forest"),
    (128, 32, 1, 16, 64, 0, "tree")])
def test_attention(lib, D, G, heads, ratio, page, window, kind, t):
    s = Trees(NARROW, heads, ratio, D, G, page, t, kind, seed=D + ratio + window, extra_words=ratio % 3, pad_rows=3)
    s.masks(window)
    assert not s.is_wide(lib)
    s.check(*s.run(lib))


@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("D,G,heads,ratio,page,window,kind", [
    (128, 128, 1, 8, 64, 0, "tree"), (128, 64, 2, 16, 32, 0, "tree"), (128, 32, 1, 16, 96, 0, "forest"), (64, 64, 2, 8, 64, 0, "chain"),
    (64, 32, 1, 16, 32, 0, "star"), (128, 64, 1, 16, 64, 33, "tree"), (64, 32, 2, 16, 32, 1, "chain"), (128, 128, 1, 16, 32, 150, "forest"),
    (128, 64, 8, 2, 64, 0, "tree")])
def test_attention_wide_tiles(lib, D, G, heads, ratio, page, window, kind, t):
    s = Trees(WIDE, heads, ratio, D, G, page, t, kind, seed=D + ratio + window, extra_words=ratio % 3, pad_rows=3)
    s.masks(window)
    most = 60000  # what the contexts may be decides about the tiles; under a window only what it leaves does
    if window:
        s.check(*s.run(lib))  # tiles of 16
        s = Trees([(17, 40 + window + i % 7) for i in range(400)], heads, ratio, D, G, page, t, kind, seed=window)
        s.masks(window)
        assert s.is_wide(lib)
        s.check(*s.run(lib))
        return
    assert s.is_wide(lib, most)
    s.check(*s.run(lib, most))


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("window", [0, 9])
def test_any_bits(lib, wide, window):
    """Masks that are no trees: rows of nothing, not even themselves, bits of nodes that there are not, and
    depths out of range."""
    spread = [(34, 34), (20, 55), (3, 40), (40, 40)] + [(12, 12 + i % 40) for i in range(200 if wide else 0)]
    s = Trees(spread, 2, 16 if wide else 2, 64, 64, 32, F16, "forest", seed=5 + window, extra_words=1)
    s.mask[:] = s.g.integers(0, 1 << 32, s.mask.shape, dtype=np.uint32)
    s.mask[::3] = 0
    s.mask[1, 0], s.mask[2] = 1 << 33 & 0xFFFFFFFF, 0xFFFFFFFF
    s.depth[:] = s.g.integers(-5, 60, s.depth.shape)
    s.depth[:4] = [2 ** 31 - 1, -2 ** 31, 33, 34]
    s.window = window
    most = 40000 if wide and not window else None
    assert s.is_wide(lib, most) == wide
    out, lse = s.run(lib, most)
    s.check(out, lse)
    assert (out[0, :s.heads * s.ratio * 64] == 0).all() and (lse[0] == -math.inf).all()


@pytest.mark.parametrize("wide", [False, True])
def test_missing_pages_and_nan_where_nobody_looks(lib, wide):
    s = Trees([(40, 96), (2, 64), (5, 3), (30, 200), (8, 8)], 1, 16 if wide else 2, 128, 64, 32, BF16, "star", seed=2)
    s.masks()
    s.table[0, 0], s.table[0, 2] = -1, 2 ** 31 - 1
    s.table[1, :2] = -1                       # nothing to see at all
    # nodes that no row names, and what lies behind the last node, hold NaN
    s.mask[s.rows[3]:s.rows[4], 0] &= np.uint32(0x0000FFFF)
    half = s.at.blocks(s.raw)[..., 32 * 128:].view(np.float16).reshape(s.pages, 1, 1, 4, 2, 32)
    slot = [8 * (t // 4 % 4) + 4 * (t // 16) + t % 4 for t in range(32)]
    for node in range(16, 30):
        p = 170 + node
        half[s.table[3, p // 32], :, :, :, :, slot[p % 32]] = np.nan
    for p in range(200, 224):
        half[s.table[3, p // 32], :, :, :, :, slot[p % 32]] = np.inf
    most = 200000 if wide else None
    assert s.is_wide(lib, most) == wide
    out, lse = s.run(lib, most)
    s.check(out, lse)
    assert (out[40:42, :128] == 0).all() and (lse[40:42] == -math.inf).all()


@pytest.mark.parametrize("t,up", [(BF16, 1e20), (BF16, 1e-20), (F16, 2e4), (F16, 1e-4)])
@pytest.mark.parametrize("wide", [False, True])
def test_query_range(lib, wide, t, up):
    s = Trees([(40, 200), (12, 12)], 1, 16 if wide else 2, 128, 64, 32, t, seed=3)
    s.masks()
    s.q = (s.q.float() * up).to(t)
    scale = 128 ** -0.5 / up if up > 1 else 128 ** -0.5
    most = 200000 if wide else None
    assert s.is_wide(lib, most) == wide
    s.check(*s.run(lib, most, scale), scale)


def test_more_columns_than_wide_tiles_have(lib):
    """700 nodes of one sequence, 16 query heads: 88 tiles of 128 columns, or 700 of 16."""
    s = Trees([(700, 1000)], 1, 16, 64, 64, 64, F16, "tree", seed=9)
    s.masks()
    s.check(*s.run(lib))
    assert s.is_wide(lib, 100000)
    s.check(*s.run(lib, 100000))


def test_many_sequences(lib):
    """More than 64, and more than 1024, which the division between workgroups goes through in turns."""
    for n, most in ((200, None), (1100, None), (1100, 8192)):
        s = Trees([(i % 5, 3 + i % 61) for i in range(n)], 1, 16, 64, 64, 32, BF16, seed=n)
        s.masks()
        s.check(*s.run(lib, most))


def test_a_chain_attends_as_tokens_in_a_row_do(lib):
    for spread, most in (([(1, 200), (20, 20), (7, 300)], None), ([(40, 200), (64, 64)], 200000)):
        s = Trees(spread, 2, 8, 128, 64, 64, F16, "chain", seed=11)
        s.masks()
        out, lse = s.run(lib, most)
        w = 16 * 128
        rows, lens, table, raw = s.dev[:4]
        o2, l2 = torch.empty_like(out), torch.empty_like(lse)
        lib.w4a16_kv4_attention(s.q.cuda(), rows, lens, table, raw, o2, l2, len(spread), s.tokens, s.max_new, s.max_len, w + 8, w + 16, 16, 2, 128,
                                64, 64, s.pages, s.width, 0, 128 ** -0.5, lib.DT_F16)
        # both are within a bound that is symmetric around the exact result: half a step and the
        # rounding of values up to 8 (2^-10 of them) each
        assert ((out[:, :w].double() - o2[:, :w].double()).abs() <= 2 * (2.0 ** -11 * o2[:, :w].double().abs() + 8 * 2.0 ** -10)).all()
        assert ((lse - l2).abs() <= 1e-4 + 2.0 ** -20 * l2.abs()).all()


@pytest.mark.parametrize("wide", [False, True])
def test_reproducible_on_streams_and_in_a_graph(lib, wide):
    s = Trees([(30, 900), (30, 1500), (30, 33), (8, 8)], 2, 16 if wide else 2, 128, 64, 64, F16, seed=12)
    s.masks()
    most = 60000 if wide else None
    assert s.is_wide(lib, most) == wide
    q = s.q.cuda()
    out0, lse0 = s.run(lib, most, q=q)
    torch.cuda.synchronize()
    w = s.heads * s.ratio * 128
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [(torch.zeros_like(out0), torch.zeros_like(lse0)) for _ in streams]
    for st, (o, l) in zip(streams, outs):  # two calls at once
        st.wait_stream(torch.cuda.current_stream())
        for _ in range(3):
            s.call(o, l, q, st)
    torch.cuda.synchronize()
    for o, l in outs:
        assert torch.equal(o[:, :w], out0[:, :w]) and torch.equal(l, lse0)
    side, (o, l) = streams[0], outs[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        s.call(o, l, q, side)
    for _ in range(3):
        q.normal_()
        s.call(out0, lse0, q, None)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o[:, :w], out0[:, :w]) and torch.equal(l, lse0)


def test_callers_workspace(lib):
    """A buffer as large as the query says serves the call; a smaller one is refused."""
    side = torch.cuda.Stream()
    for ratio, most in ((2, None), (16, 60000)):
        s = Trees([(30, 900), (30, 1500)], 2, ratio, 128, 64, 64, F16, seed=13)
        s.masks()
        out, lse = s.run(lib, most)
        torch.cuda.synchronize()
        need = lib.w4a16_kv4_tree_workspace_bytes(2, s.tokens, 30, most or 1500, 2 * ratio, 2, 128, 0)
        size = lib.WS_COUNTER_BYTES + need
        buf = torch.empty(size + 1024, dtype=torch.uint8, device="cuda")
        at = (buf.data_ptr() + 255) // 256 * 256
        buf[-512:] = 99
        o, l = torch.zeros_like(out), torch.zeros_like(lse)
        q = s.q.cuda()
        torch.cuda.synchronize()
        try:
            lib.w4a16_set_workspace(at, size, side)
            s.call(o, l, q, side)
            side.synchronize()
            assert torch.equal(o[:, :2 * ratio * 128], out[:, :2 * ratio * 128]) and torch.equal(l, lse)
            lib.w4a16_set_workspace(at, size - 2048 - 256, side)  # without what the query says of counters, and 256
            with pytest.raises(lib.W4A16Error) as e:
                s.call(o, l, q, side)
            assert e.value.code == -6
        finally:
            lib.w4a16_set_workspace(None, 0, side)


@pytest.mark.parametrize("ratio,most", [(2, None), (16, 60000)])
def test_pages_past_4_gib(lib, ratio, most):
    """The same pages at the end of a cache of 5 GiB give the same bits."""
    s = Trees([(40, 200), (30, 90)], 8, ratio, 128, 64, 64, F16, seed=14)
    s.masks()
    out, lse = s.run(lib, most)
    size = s.raw.shape[1]
    pages = (5 << 30) // size
    big = torch.zeros(pages, size, dtype=torch.uint8, device="cuda")
    big[pages - s.pages:] = s.dev[3]
    table = torch.where(s.dev[2] >= 0, s.dev[2] + (pages - s.pages), -1).to(torch.int32)
    w = 8 * ratio * 128
    o, l = torch.zeros_like(out), torch.zeros_like(lse)
    lib.w4a16_kv4_tree_attention(s.q.cuda(), s.dev[0], s.dev[1], table, big, s.dev[4], None, o, l, 2, s.tokens, s.max_new, most or s.max_len, s.words,
                                 w + 8, w + 16, 8 * ratio, 8, 128, 64, 64, pages, s.width, 0, 128 ** -0.5)
    assert torch.equal(o[:, :w], out[:, :w]) and torch.equal(l, lse)


@pytest.mark.parametrize("D", [64, 128])
def test_one_call_covers_the_captures_of_others(lib, D):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s = Trees([(2, 9)], 1, 1, D, 64, 32, F16, seed=15)
    s.masks()
    s.run(lib, stream=side)
    for spread, heads, ratio, most in (([(40, 900)], 2, 4, None), ([(60, 900), (33, 200)], 2, 16, 60000), ([(7, 900)], 4, 1, 4000)):
        s = Trees(spread, heads, ratio, D, 64, 64, F16, seed=16)
        s.masks()
        out, lse = s.run(lib, most)
        q, w = s.q.cuda(), heads * ratio * D
        o, l = torch.zeros_like(out), torch.zeros_like(lse)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            s.call(o, l, q, side)  # refused if the stream holds too little
        for _ in range(2):
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(o[:, :w], out[:, :w]) and torch.equal(l, lse)
