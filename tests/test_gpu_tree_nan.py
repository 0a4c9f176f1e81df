"""GPU tests of NaN in trees of drafted tokens: a NaN of a node's keys or values reaches the nodes that see it
(its branch below it) and no others; the rest stays within the bounds of tests/tree_ref.py."""
import math

import numpy as np
import pytest
import torch

import decoder_ref as ref
import tree_ref as tr
from test_gpu_tree import BF16, F16, Trees

pytestmark = pytest.mark.gpu


def spoil(s, b, position, which, group, word):
    """NaN in the s (0) or m (1) of a group of a token's K (0) or V (1), in every head."""
    half = s.at.blocks(s.raw)[..., 32 * s.D:].view(np.float16).reshape(s.pages, s.heads, s.page // 32, 2 * s.D // s.G, 2, 32)
    t = position % 32
    half[s.table[b, position // s.page], :, position % s.page // 32, which * (s.D // s.G) + group, word, 8 * (t // 4 % 4) + 4 * (t // 16) + t % 4] = np.nan


def check(s, out, lse):
    """A row that sees NaN keys is NaN; one that sees NaN values is NaN in their channels; else as without them."""
    out, lse, vals, step = out.cpu(), lse.cpu().double(), s.at.values(s.raw), ref.half_step(s.t)
    reached = [0, 0, 0]
    for b, (n, L) in enumerate(s.spread):
        seen, page, place = s.seen(b)
        mine = slice(s.rows[b], s.rows[b + 1])
        for h in range(s.heads * s.ratio):
            k, v = (torch.from_numpy(vals[i, page, h // s.ratio, place]) for i in (0, 1))
            o, l, otol, ltol = tr.attend(s.q[mine, h * s.D:(h + 1) * s.D].double(), k.nan_to_num(0.0), v.nan_to_num(0.0), seen, s.D ** -0.5)
            rows = (seen.double() @ k.isnan().any(1).double()) > 0
            bad = ((seen.double() @ v.isnan().double()) > 0) | rows[:, None]
            got = out[mine, h * s.D:(h + 1) * s.D].double()
            assert torch.equal(got.isnan(), bad), (b, h)
            assert torch.equal(lse[mine, h].isnan(), rows), (b, h)
            off = (got - o).abs()
            assert (off <= step * o.abs() + otol * (1 + step) + 2.0 ** -25)[~bad].all(), (b, h)
            none = l == -math.inf  # a row that sees nothing
            assert torch.equal(lse[mine, h][~rows] == -math.inf, none[~rows]), (b, h)
            assert ((lse[mine, h] - l).abs() <= ltol)[~rows & ~none].all(), (b, h)
            reached = [reached[0] + int(rows.sum()), reached[1] + int((bad.any(1) & ~rows).sum()), reached[2] + int((~bad.any(1)).sum())]
    return reached


@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("D,G,heads,ratio,page,kind", [
    (128, 128, 2, 1, 64, "tree"), (128, 64, 1, 3, 32, "star"), (128, 32, 1, 2, 96, "forest"), (64, 64, 1, 2, 64, "tree"), (64, 32, 2, 1, 32, "star")])
@pytest.mark.parametrize("wide", [False, True])
def test_nan_of_a_branch(lib, wide, D, G, heads, ratio, page, kind, t):
    ratio *= 8 if wide else 1
    spread = [(40, 96), (20, 900), (33, 33), (7, 71)]
    s = Trees(spread, heads, ratio, D, G, page, t, kind, seed=D + G)
    s.masks()
    g, ng = np.random.default_rng(3), D // G
    for b, (n, L) in enumerate(spread):
        for j in (1, 3, n // 2, n - 1):
            spoil(s, b, L - n + j, 1, int(g.integers(ng)), int(g.integers(2)))
    spoil(s, 0, 96 - 40 + 11, 0, 0, 0)       # keys
    spoil(s, 2, 30, 0, ng - 1, 1)
    spoil(s, 3, 71 - 7 + 2, 1, 0, 0)         # several groups of one token
    spoil(s, 3, 71 - 7 + 2, 1, ng - 1, 1)
    most = 200000 if wide else None
    assert s.is_wide(lib, most) == wide
    assert min(check(s, *s.run(lib, most))) > 0


@pytest.mark.parametrize("ratio", [1, 8])
def test_nan_in_tiles_of_8_columns(lib, ratio):
    new = 8 // ratio
    s = Trees([(new, 50), (new, 700), (max(1, new - 1), 33)], 2, ratio, 128, 32, 32, F16, "star", seed=4)
    s.masks()
    for b, (n, L) in enumerate(s.spread):
        if n > 1:
            spoil(s, b, L - 1, 1, 3, 1)
            spoil(s, b, L - n + 1, 1, 1, 0)
    if ratio == 8:
        s.mask[0] = 0                        # its own NaN, which it does not see
        spoil(s, 0, 49, 1, 0, 0)
    assert not s.is_wide(lib)
    assert check(s, *s.run(lib))[2] > 0


@pytest.mark.parametrize("wide", [False, True])
def test_nan_of_a_token_that_only_some_windows_reach(lib, wide):
    """Held tokens that shallow nodes see and deep ones do not."""
    if wide:
        s = Trees([(17, 60 + i % 7) for i in range(400)], 1, 16, 64, 32, 32, BF16, "chain", seed=5)
    else:
        s = Trees([(17, 60), (30, 300)], 1, 2, 64, 32, 32, F16, "chain", seed=5)
    s.masks(12)
    for b, (n, L) in enumerate(s.spread):
        spoil(s, b, L - n - 9, 1, b % 2, 0)
    assert s.is_wide(lib) == wide
    reached = check(s, *s.run(lib))
    assert reached[1] > 0 and reached[2] > 0


@pytest.mark.parametrize("wide", [False, True])
def test_all_nodes_nan_and_any_bits(lib, wide):
    """Every node's values NaN in one group; rows that name none of them, and rows with random bits."""
    s = Trees([(40, 200), (25, 25), (10, 1000)], 1, 16 if wide else 2, 128, 64, 64, F16, "forest", seed=6, extra_words=1)
    s.mask[:] = s.g.integers(0, 1 << 32, s.mask.shape, dtype=np.uint32) & s.g.integers(0, 1 << 32, s.mask.shape, dtype=np.uint32)
    s.mask[::3] = 0
    for b, (n, L) in enumerate(s.spread):
        for j in range(n):
            spoil(s, b, L - n + j, 1, j % 2, j // 2 % 2)
    most = 200000 if wide else None
    assert s.is_wide(lib, most) == wide
    out, lse = s.run(lib, most)
    reached = check(s, out, lse)
    assert reached[1] > 0 and reached[2] > 0
    assert not out.cpu()[0, :s.heads * s.ratio * 128].isnan().any() and math.isfinite(float(lse[0, 0]))
