"""The classes around drafted trees (decoder.py): refusals on the host (CPU); a search with drafted trees
over several layers, step after step, against the same tokens decoded one by one; and the attention block
with a tree against its parts (GPU)."""
import math

import pytest
import torch

import tree_ref as tr


def test_refusals_on_the_host():
    pytest.importorskip("w4a16_mixed_precision_offline_amd")
    from w4a16_mixed_precision_offline_amd.decoder import Batch, Kv4Cache, Kv4Pool, Rotary, Tree
    i32 = lambda *x: torch.zeros(x, dtype=torch.int32)  # noqa: E731
    h = lambda *x: torch.zeros(x, dtype=torch.float16)  # noqa: E731
    b = Batch(i32(3), i32(2), i32(2, 2), 1, 32)
    for bad in (i32(2, 2), torch.zeros(4, dtype=torch.int64)):
        with pytest.raises(ValueError):
            Tree(bad, b)
    with pytest.raises(ValueError):
        Tree(i32(4), b)  # host tensors
    empty = Tree(i32(0), b)
    assert empty.mask.shape == (0, 1)
    for freq, head in ((torch.ones(4), 64), (torch.ones(12), 64), (torch.ones(40), 64), (torch.ones(8), 20), (torch.ones(8), 1024)):
        with pytest.raises(ValueError):
            Rotary(freq, head)
    with pytest.raises(TypeError):
        Rotary(torch.ones(8).half(), 64)
    with pytest.raises(ValueError):
        Rotary(torch.ones(8), 64, i32(9))
    r = Rotary(torch.ones(8), 64).half()
    assert r.freq.dtype == torch.float32 and not r.double().freq.dtype == torch.float64
    for q, k, pos in ((h(3, 64), h(3, 64), i32(2)), (h(3, 65), None, i32(3)), (h(3, 64), h(2, 64), i32(3)), (h(3, 64), h(3, 64), i32(2, 3)),
                      (h(3, 64), h(3, 64).bfloat16(), i32(3)), (h(64, 3).t(), None, i32(3)), (h(3, 64), None, i32(3))):
        with pytest.raises(ValueError):
            r(q, k, pos)
    with pytest.raises(TypeError):
        r(torch.zeros(3, 64), None, i32(3))
    r.freq = r.freq.half()
    with pytest.raises(TypeError):
        r(h(3, 64), None, i32(3))
    for bad in (dict(layers=0), dict(pages=0), dict(head=96), dict(page=48)):
        with pytest.raises(ValueError):
            Kv4Pool(**{**dict(layers=2, pages=4, kv_heads=1, head=64, device="cpu"), **bad})
    pool = Kv4Pool(2, 4, 1, 64, 64, 32, device="cpu")
    assert len(pool) == 2 and not pool.state_dict()
    pool.data.fill_(7)
    assert (pool[1].data == 7).all() and pool[1].data.data_ptr() == pool.data[1].data_ptr()
    pool.half().double()  # a cast leaves codes alone, and the layers stay the pool's
    assert pool[0].data.data_ptr() == pool.data.data_ptr() and pool.data.dtype == torch.uint8
    with pytest.raises(ValueError):
        Kv4Cache(4, 1, 64, 64, 32, data=torch.zeros(4, 7, dtype=torch.uint8))
    with pytest.raises(ValueError):
        pool[0].attend_tree(h(2, 64), b, empty, 1)
    for path, count in ((i32(2), i32(2)), (i32(3, 2), i32(2)), (i32(2, 2), i32(3)), (i32(2, 2).long(), i32(2)), (i32(2, 2), i32(2))):
        with pytest.raises(ValueError):
            pool.compact(path, count, b)
    for args in ((i32(2), i32(2), i32(2)), (i32(2, 2), i32(3), i32(2)), (i32(2, 2), i32(2), i32(0)), (i32(2, 2), i32(2), i32(2), i32(3)),
                 (i32(2, 2), i32(2), i32(2), None, None, i32(4)), (i32(2, 2), i32(2), i32(2))):
        with pytest.raises(ValueError):
            pool.fork(*args)


@pytest.mark.gpu
def test_a_search_with_trees(lib):
    """Two requests with two beams each over two layers: every step drafts a tree for each beam, turns
    queries and keys by the nodes' positions on three axes, appends, attends, keeps a branch, moves its tokens and forks
    the beams.  What each node attends to is the same as for tokens decoded one by one on a sequence of their own."""
    from w4a16_mixed_precision_offline_amd.decoder import Batch, Kv4Pool, Rotary, Tree
    import random
    r, g = random.Random(1), torch.Generator().manual_seed(1)
    L, heads, kv, D, page, pages = 2, 8, 2, 64, 32, 60
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pool, plain = Kv4Pool(L, pages, kv, D, 32, page), Kv4Pool(L, pages, kv, D, 32, page)
    rotary = Rotary(1000.0 ** (-torch.arange(32, dtype=torch.float32) / 32).cuda(), D, i32([i % 3 for i in range(32)]))
    width = (heads + 2 * kv) * D
    new = lambda n: torch.randn(L, n, width, generator=g).half().cuda()  # noqa: E731
    axes = lambda pos: torch.stack([pos, pos // 3, pos % 7]).contiguous()  # noqa: E731

    def put(pool, x, batch, pos):
        out = []
        for i in range(L):
            q, k, v = x[i].split([heads * D, kv * D, kv * D], 1)
            rotary(q, k, axes(pos))
            pool[i].append(k, v, batch)
            out.append(q)
        return out

    # prompts: both beams of a request go on from one sequence
    lens = [40, 75]
    table, held, missing = pool.fork(torch.full((2, 8), -1, dtype=torch.int32, device="cuda"), i32([0, 0]), i32([-1, -1]), None, i32(lens))
    assert missing.item() == 0 and held.tolist() == [0, 0]
    x = new(sum(lens))
    put(pool, x, Batch(i32([0, 40, 115]), i32(lens), table, 75, 75), i32(list(range(40)) + list(range(75))))
    story = [[x[:, a:a + 1].clone() for a in range(o, o + n)] for o, n in ((0, 40), (40, 75))]  # each sequence's turned rows
    story = [story[0], list(story[0]), story[1], list(story[1])]
    parent, lens = [0, 0, 1, 1], i32(lens)
    for step in range(4):
        sizes = [r.randint(4, 9) for _ in range(4)]
        now = [len(s) for s in story]
        before = lens
        table, lens, missing = pool.fork(table, before, i32(parent), None, i32([a + n for a, n in zip(now, sizes)]))
        assert missing.item() == 0 and lens.tolist() == now
        parents = [tr.trees(r, "forest" if step % 2 else "tree", n) for n in sizes]
        rows = [0]
        for n in sizes:
            rows.append(rows[-1] + n)
        batch = Batch(i32(rows), i32([a + n for a, n in zip(now, sizes)]), table, max(sizes), 200)
        tree = Tree(i32([p for t in parents for p in t]), batch)
        x = new(rows[-1])
        q = put(pool, x, batch, tree.pos)
        out = [pool[i].attend_tree(q[i], batch, tree, heads) for i in range(L)]
        paths = []
        for b in range(4):
            lines = tr.branches(parents[b])
            for j in (0, sizes[b] - 1, r.randrange(sizes[b])):
                # the node's line behind the story, on pages of its own, its last token attending to it all
                line = lines[j][::-1]
                rws = torch.cat(story[b] + [x[:, rows[b] + i:rows[b] + i + 1] for i in line], 1)
                n = rws.shape[1]
                one = Batch(i32([0, n]), i32([n]), torch.arange(8, dtype=torch.int32, device="cuda").view(1, 8), n, n)
                for i in range(L):
                    _, k, v = rws[i].split([heads * D, kv * D, kv * D], 1)
                    plain[i].append(k, v, one)
                    last = Batch(i32([0, 1]), i32([n]), one.table, 1, n)
                    want = plain[i].attend(rws[i, -1:, :heads * D], last, heads)
                    # two results of one formula, each off by half a step of its own and by two
                    # roundings of values up to 6 (a code's value, the probability)
                    off = (out[i][rows[b] + j].double() - want[0].double()).abs()
                    assert (off <= 2 * (2.0 ** -11 * want[0].double().abs() + 6 * 2.0 ** -10)).all(), (step, b, j)
            paths.append(lines[r.randrange(sizes[b])][::-1])
        most = max(len(p) for p in paths)
        lens = pool.compact(i32([p + [-1] * (most - len(p)) for p in paths]), i32([len(p) for p in paths]), batch)
        assert lens.tolist() == [a + len(p) for a, p in zip(now, paths)]
        for b, p in enumerate(paths):
            story[b] = story[b] + [x[:, rows[b] + i:rows[b] + i + 1].clone() for i in p]
        # the whole sequences read back are what one that was never drafted holds
        n = [len(s) for s in story]
        at = [0]
        for a in n:
            at.append(at[-1] + a)
        whole = Batch(i32(at), lens, table, max(n), max(n))
        for i in range(L):
            k, v = (torch.empty(at[-1], kv * D, dtype=torch.float16, device="cuda") for _ in range(2))
            pool[i].gather(k, v, whole)
            for b in range(4):
                rws = torch.cat(story[b], 1)[i]
                one = Batch(i32([0, n[b]]), i32([n[b]]), torch.arange(8, dtype=torch.int32, device="cuda").view(1, 8), n[b], n[b])
                plain[i].append(*rws.split([heads * D, kv * D, kv * D], 1)[1:], one)
                k2, v2 = (torch.empty(n[b], kv * D, dtype=torch.float16, device="cuda") for _ in range(2))
                plain[i].gather(k2, v2, one)
                assert torch.equal(k[at[b]:at[b + 1]], k2) and torch.equal(v[at[b]:at[b + 1]], v2), (step, i, b)
        parent = [0, 0, 2, 3] if step % 2 else [1, 0, 3, 3]
        story = [story[p] for p in parent]


@pytest.mark.gpu
def test_block_with_a_tree(lib):
    from w4a16_mixed_precision_offline_amd.decoder import AttentionBlock, Batch, Kv4Cache, Rotary, Tree
    from w4a16_mixed_precision_offline_amd.layer import W4A16Linear
    K, heads, kv, D, page = 256, 4, 2, 64, 32
    g = torch.Generator().manual_seed(2)

    def linear(k, n):
        q = torch.randint(-2 ** 31, 2 ** 31 - 1, (k // 8, n), generator=g, dtype=torch.int32)
        return W4A16Linear.from_quantized(q.cuda(), (torch.rand(k // 128, n, generator=g) * 0.01 + 0.002).half().cuda())

    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = Kv4Cache(8, kv, D, 32, page)
    block = AttentionBlock(torch.ones(K).half().cuda(), linear(K, (heads + 2 * kv) * D), linear(heads * D, K), cache, heads)
    rotary = Rotary(100.0 ** (-torch.arange(16, dtype=torch.float32) / 16).cuda(), D, neighbours=True)
    x = torch.randn(50, K, generator=g).half().cuda()
    table = i32([[3, 5, 1]])
    first = Batch(i32([0, 50]), i32([50]), table, 50, 50)
    block(x, None, first, rotate=rotary.at(i32(list(range(50)))))
    batch = Batch(i32([0, 6]), i32([56]), table, 6, 56)
    for window in (0, 3):
        tree = Tree(i32([-1, 0, 0, 1, 3, 2]), batch, window)
        assert tree.pos.tolist() == [50, 51, 51, 52, 53, 52]
        with pytest.raises(ValueError):
            block(x[:6], None, batch, tree=tree, window=window + 1)
        y, _ = block(x[:6], None, batch, window=window, rotate=rotary.at(tree.pos), tree=tree)
        # part by part
        h, y8 = torch.empty(6, K, dtype=torch.float16, device="cuda"), torch.empty(6, K, dtype=torch.float8_e4m3fn, device="cuda")
        s = torch.empty(6, device="cuda")
        lib.w4a8_rmsnorm(x, None, block.gamma, h, y8, s, None, 6, K, 1e-5)
        qkv = block.qkv(y8, s)
        q, k, v = qkv.split([heads * D, kv * D, kv * D], 1)
        rotary(q, k, tree.pos)
        cache.append(k, v, batch)
        lse = torch.zeros(6, heads, device="cuda")
        o = cache.attend_tree(q, batch, tree, heads, lse=lse)
        assert torch.equal(y, block.out(o)) and lse.isfinite().all()
    q = q.contiguous().float().half().requires_grad_()
    with pytest.raises(ValueError):
        rotary(q, None, tree.pos)
    with torch.no_grad():
        rotary(q, None, tree.pos)
    assert math.isfinite(float(y.float().abs().max()))


@pytest.mark.gpu
def test_padding_rows_and_padded_trees(lib):
    """Rows of no sequence, as a batch padded for a graph has them: 0 out of attend_tree, whatever the
    tree says of them."""
    from w4a16_mixed_precision_offline_amd.decoder import Batch, Kv4Pool, Tree
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pool = Kv4Pool(1, 4, 1, 64, 64, 32)
    q = torch.randn(9, 128, device="cuda").half()
    k, v = torch.randn(9, 64, device="cuda").half(), torch.randn(9, 64, device="cuda").half()
    batch = Batch(i32([0, 3, 5]), i32([3, 2]), i32([[0], [1]]), 3, 32)
    tree = Tree(i32([-1, 0, 0, -1, 0, 5, 5, 5, 5]), batch)
    assert (tree.mask[5:] == 0).all() and tree.pos[:5].tolist() == [0, 1, 1, 0, 1]
    pool[0].append(k, v, batch)
    out = pool[0].attend_tree(q, batch, tree, 2)
    assert (out[5:] == 0).all() and (out[:5] != 0).any(1).all()
