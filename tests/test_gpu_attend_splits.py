"""GPU tests of how attention over the 4-bit cache is divided: stripes over many sequences,
tiles shared by workgroups, long contexts, against the formula in 64 bits."""
import math

import numpy as np
import pytest
import torch

import decoder_ref as ref

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


class Case:
    def __init__(self, w4, spread, heads, ratio, D, G, page, t, seed=0, shared=False):
        self.w4, self.spread, self.heads, self.ratio, self.D, self.G, self.page, self.t = w4, spread, heads, ratio, D, G, page, t
        g = torch.Generator().manual_seed(seed)
        used = [max(0, -(-L // page)) for _, L in spread]
        self.width = max(used) + 1
        self.pages = (max(used) if shared else sum(used)) + 2
        order = torch.randperm(self.pages, generator=g).tolist()
        self.table = torch.full((len(spread), self.width), -1, dtype=torch.int32)
        at = 0
        for b, u in enumerate(used):
            self.table[b, :u] = torch.tensor(order[at:at + u], dtype=torch.int32)
            at += 0 if shared else u
        self.rows = [0]
        for n, _ in spread:
            self.rows.append(self.rows[-1] + n)
        self.lens = [L for _, L in spread]
        self.tokens = self.rows[-1]
        size = w4.w4a16_kv4_page_bytes(heads, D, G, page)
        blocks = heads * (page // 32)
        raw = torch.randint(0, 256, (self.pages, blocks, size // blocks), generator=g, dtype=torch.uint8)
        # s in 2^-4 .. 2^-2 and m in -2 .. 2 at every place
        par = torch.empty(self.pages, blocks, 2, D // G, 2, 32, dtype=F16)
        par[..., 0, :] = torch.rand(par[..., 0, :].shape, generator=g) * 0.1875 + 0.0625
        par[..., 1, :] = torch.rand(par[..., 1, :].shape, generator=g) * 4 - 2
        raw[..., 32 * D:] = par.flatten(2).view(torch.uint8)
        self.raw = raw.view(self.pages, size)
        self.q = torch.randn(self.tokens, heads * ratio * D, generator=g).to(t)

    def run(self, window=0, max_len=None, table=None, lens=None, twice=True):
        d = lambda x: torch.as_tensor(x, dtype=torch.int32).cuda()  # noqa: E731
        self.now_table = self.table if table is None else table
        self.now_lens = self.lens if lens is None else lens
        args = [d(self.rows), d(self.now_lens), d(self.now_table), self.raw.cuda()]
        q, outs = self.q.cuda(), []
        hd = self.heads * self.ratio * self.D
        for _ in range(2 if twice else 1):  # the second call finds the workspace as the first left it
            out = torch.full((self.tokens, hd), math.nan, dtype=self.t, device="cuda")
            lse = torch.full((self.tokens, self.heads * self.ratio), math.nan, device="cuda")
            self.w4.w4a16_kv4_attention(q, *args, out, lse, len(self.spread), self.tokens, max(n for n, _ in self.spread),
                                        max_len or max(self.lens), hd, hd, self.heads * self.ratio, self.heads, self.D, self.G,
                                        self.page, self.pages, self.width, window, self.D ** -0.5,
                                        self.w4.DT_BF16 if self.t == BF16 else self.w4.DT_F16)
            outs.append((out.cpu(), lse.cpu()))
        if twice:
            assert torch.equal(outs[0][0].view(torch.int16), outs[1][0].view(torch.int16))
            assert torch.equal(outs[0][1].view(torch.int32), outs[1][1].view(torch.int32))
        return outs[0]

    def held(self, b, h, length):
        """Keys and values [length, D] of sequence b, kv head h, and which have a page."""
        D, G, P = self.D, self.G, self.page
        p = np.arange(length)
        pages = self.now_table[b].numpy()[p // P]
        have = (pages >= 0) & (pages < self.pages)
        blocks = self.raw.view(self.pages, self.heads, P // 32, -1).numpy()[np.where(have, pages, 0), h, p % P // 32]
        t, d = p % 32, np.arange(D)
        e = d % 8
        nib = e // 2 + 4 * (e % 2)
        word = (t[:, None] // 16 * 64 + d // 8 % 4 * 16 + t[:, None] % 16) * (D // 32) + d // 32
        i = np.arange(length)[:, None]
        k = (blocks[i, 4 * word + nib // 2] >> (4 * (nib % 2))) & 15
        e = 4 * (t // 16) + t % 4
        nib = (e // 2 + 4 * (e % 2))[:, None]
        word = (d // 64 * 64 + t[:, None] // 4 % 4 * 16 + d % 16) * 4 + d // 16 % 4
        v = (blocks[i, 16 * D + 4 * word + nib // 2] >> (4 * (nib % 2))) & 15
        par = np.ascontiguousarray(blocks[:, 32 * D:]).view(np.float16).reshape(length, 2, D // G, 2, 32).astype(np.float64)
        slot = 8 * (t // 4 % 4) + 4 * (t // 16) + t % 4
        s, m = (par[np.arange(length), :, :, w, slot].repeat(G, axis=2) for w in (0, 1))  # [length, K or V, D]
        return torch.from_numpy(m[:, 0] + s[:, 0] * k), torch.from_numpy(m[:, 1] + s[:, 1] * v), torch.from_numpy(have)

    def check(self, out, lse, window=0, seqs=None, heads=None, rows=None):
        step = ref.half_step(self.t)
        D = self.D
        for b in range(len(self.spread)) if seqs is None else seqs:
            n, L = self.spread[b][0], min(self.now_lens[b], self.width * self.page)
            first = self.now_lens[b] - n
            for h in range(self.heads) if heads is None else heads:
                if L > 0:
                    k, v, have = self.held(b, h, L)
                else:
                    k, v, have = torch.zeros(0, D).double(), torch.zeros(0, D).double(), torch.zeros(0, dtype=torch.bool)
                pos = torch.arange(max(L, 0))
                for i in range(n) if rows is None else [x for x in rows if x < n]:
                    seen = have & (pos <= first + i) & (pos > first + i - window if window else True)
                    for c in range(self.ratio):
                        hq = h * self.ratio + c
                        q = self.q[self.rows[b] + i, hq * D:(hq + 1) * D].double()
                        o, l, otol, ltol = ref.attend(q, k, v, seen, D ** -0.5, self.t)
                        got = out[self.rows[b] + i, hq * D:(hq + 1) * D].double()
                        err = (got - o).abs()
                        assert (err <= step * o.abs() + otol * (1 + step) + 2.0 ** -25).all(), (b, i, hq, float((err - otol).max()))
                        g = float(lse[self.rows[b] + i, hq])
                        assert g == l if l == -math.inf else abs(g - l) <= ltol, (b, i, hq, g, l, ltol)


@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("heads,ratio,D,G,page", [(2, 8, 128, 32, 64), (1, 1, 128, 128, 32), (3, 5, 64, 64, 96), (1, 16, 128, 64, 64),
                                                  (2, 12, 64, 32, 32)])
def test_one_long_sequence(lib, heads, ratio, D, G, page, t):
    c = Case(lib, [(1, 40001)], heads, ratio, D, G, page, t)
    c.check(*c.run())
    c.check(*c.run(30000), window=30000)
    c.check(*c.run(200), window=200)


@pytest.mark.parametrize("heads,ratio,D,G,t", [(2, 4, 128, 64, F16), (8, 1, 64, 32, BF16)])
def test_many_sequences_of_one_token(lib, heads, ratio, D, G, t):
    """Stripes of several tiles, tiles of several stripes, sequences without new tokens; more
    than 64 sequences take the scan in groups."""
    g = np.random.default_rng(3)
    for batch in (5, 63, 70, 200):
        spread = [(int(g.random() < 0.9), int(g.integers(1, 40) if b % 3 else g.integers(1, 9000))) for b in range(batch)]
        spread[0] = (1, 9001)
        c = Case(lib, spread, heads, ratio, D, G, 64, t, seed=batch, shared=True)
        c.check(*c.run(), seqs=sorted({0, 1, 2, 3, 4} | {b for b in (30, 62, 63, 64, 65, 127, 128, 199) if b < batch}))


def test_more_sequences_than_the_scan_takes(lib):
    g = np.random.default_rng(4)
    c = Case(lib, [(1, int(x)) for x in g.integers(1, 700, 1100)], 1, 2, 64, 64, 32, F16, shared=True)
    c.check(*c.run(), seqs=[0, 1, 7, 8, 500, 1023, 1024, 1099])


@pytest.mark.parametrize("t", [F16, BF16])
def test_a_few_new_tokens(lib, t):
    for ratio, new in ((4, 2), (4, 3), (2, 17), (16, 4)):  # 8, 12, 34 and 64 columns
        c = Case(lib, [(new, 7000), (1, 3), (new, new), (new - 1, 333)], 2, ratio, 128, 64, 64, t, seed=new)
        c.check(*c.run())
        c.check(*c.run(100), window=100)


@pytest.mark.parametrize("heads,ratio,D,G,page,t", [(1, 4, 128, 128, 64, F16), (2, 2, 128, 64, 32, BF16), (1, 8, 128, 32, 96, F16),
                                                    (2, 1, 64, 64, 64, F16), (1, 3, 64, 32, 32, BF16)])
def test_tiles_of_128_columns_in_chunks(lib, heads, ratio, D, G, page, t):
    new = 150 // ratio
    c = Case(lib, [(new, 9000), (3, 40), (0, 9), (new, new), (new // 2, 4999)], heads, ratio, D, G, page, t)
    rows = [0, 1, 2, new // 3, new // 2, new - 1]
    c.check(*c.run(), rows=rows, heads=[0])
    c.check(*c.run(1500), window=1500, rows=rows, heads=[0])
    # the same without chunks
    out, lse = c.run(max_len=1)
    c.check(out, lse, rows=rows, heads=[0])


def test_tiles_of_128_columns_whole(lib):
    spread = [(40 + 3 * b, 300 + 70 * b) for b in range(18)]
    c = Case(lib, spread, 8, 16, 64, 64, 64, F16, shared=True)  # more tiles than chunks are cut for
    c.check(*c.run(), rows=[0, 13, 39], heads=[0, 7], seqs=[0, 9, 17])


def test_missing_pages_in_shared_tiles(lib):
    for new in (1, 80):
        c = Case(lib, [(new, 20000), (new, 700)], 1, 2, 128, 64, 64, F16)
        table = c.table.clone()
        table[0, 20:200] = -1
        table[0, 251] = c.pages
        table[1, :] = 2 ** 31 - 1
        out, lse = c.run(table=table)
        c.check(out, lse, rows=[0, 1, new - 1])
        assert (out[new:] == 0).all() and (lse[new:] == -math.inf).all()


def test_lengths_past_every_page(lib):
    """A length far past the table: what has a page is seen, the rest is not there."""
    for new in (1, 80):
        c = Case(lib, [(new, 5000), (new, 300)], 1, 2, 128, 64, 64, F16)
        c.check(*c.run(lens=[2 ** 31 - 1, 300]), rows=[0, new - 1])
        c.check(*c.run(lens=[-5, 300]), rows=[0, new - 1])


def test_rows_that_overlap_leave_the_workspace_as_it_was(lib):
    """Rows that run backwards ask for more tiles than there are tokens: such a call writes no
    place but its outputs', and the next call is right."""
    for new, ratio in ((1, 8), (40, 4)):
        c = Case(lib, [(new, 6000)] * 6, 2, ratio, 128, 64, 64, F16, shared=True)
        right = c.run()
        rows, c.rows = c.rows, [0, c.tokens, 0, c.tokens, 0, c.tokens, 0]
        c.run(twice=False)
        c.rows = rows
        again = c.run()
        assert torch.equal(right[0], again[0]) and torch.equal(right[1], again[1])
        c.check(*again, rows=[0, new - 1], seqs=[0, 5])


def test_graph_replays_of_shared_tiles(lib):
    c = Case(lib, [(1, 20000), (1, 77), (1, 5000)], 2, 8, 128, 64, 64, F16)
    want = c.run()
    d = lambda x: torch.as_tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    q, rows, lens, table, raw = c.q.cuda(), d(c.rows), d(c.lens), d(c.table), c.raw.cuda()
    out, lse = torch.empty_like(q), torch.empty(3, 16, device="cuda")
    st = torch.cuda.Stream()

    def call():
        lib.w4a16_kv4_attention(q, rows, lens, table, raw, out, lse, 3, 3, 1, 20000, 2048, 2048, 16, 2, 128, 64, 64, c.pages,
                                c.width, 0, 128 ** -0.5, lib.DT_F16)
    with torch.cuda.stream(st):
        call()
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        call()
    for _ in range(4):
        out.zero_()
        lse.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), want[0]) and torch.equal(lse.cpu(), want[1])
        eager = c.run()  # other work in between, on another stream's workspace
        assert torch.equal(eager[0], want[0])
