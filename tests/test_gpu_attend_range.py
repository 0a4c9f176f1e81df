"""GPU tests of attention over the 4-bit cache where logits are far from 0: queries near the end
of their type's range, all logits far below 0, in tiles of 8, 16 and 128 columns."""
import numpy as np
import pytest
import torch

import decoder_ref as ref
from test_gpu_decoder_ops import BF16, F16, Setup

pytestmark = pytest.mark.gpu
# new tokens of a sequence of 700 (shared by workgroups) and one of 90, two query heads a kv head
TILES = {"8": (1, 1), "16": (8, 3), "128": (70, 70)}


def one_hot(lib, tile, t, D, G, q, k, scale=None):
    """Keys of one sign whose means lie apart: one key has all the weight, so a row of out is
    its value (rounded to fp16, then to t) and lse its logit."""
    n0, n1 = TILES[tile]
    s = Setup([(n0, 700), (n1, 90)], 1, D, G, 64, t, q_heads=2, seed=len(tile) + D)
    g = np.random.default_rng(5)
    for b, (_, L) in enumerate(s.spread):
        for p, a in enumerate(g.permutation(np.linspace(0.5, 1.5, L))):
            keys = (a + 0.01 * g.standard_normal((1, D))) * k
            pg = s.table[b, p // 64]
            s.model.put(pg, p % 64, keys.astype(np.float32), g.standard_normal((1, D)).astype(np.float32))
            s.model.write(s.raw, pg, p % 64)
    s.qkv[:, :2 * D] = (q * (1 + 0.01 * s.qkv[:, :2 * D].float().clamp(-3, 3))).to(t)
    s.device()
    scale = scale or D ** -0.5
    out, lse = s.attend(lib, 0, scale)
    out, lse = out.cpu().double(), lse.cpu().double()
    for b, (n, L) in enumerate(s.spread):
        vals = torch.from_numpy(np.stack([s.model.values(s.table[b, p // 64], p % 64) for p in range(L)]))[:, :, 0]
        for i in [i for i in (0, 1, 7, 31, 33, 69) if i < n]:
            row, seen = s.rows[b] + i, L - n + i + 1
            for h in range(2):
                x = vals[:seen, 0] @ s.qkv[row, h * D:(h + 1) * D].double() * scale
                first, second = x.topk(2).values.tolist()
                # sums of D products and D / G scalings in fp32 cannot take the first place from it
                assert abs(first) < 3e38 / 1.45 and first - second > 4 * (D + 8) * 2.0 ** -24 * abs(first) + 100
                want = vals[int(x.argmax()), 1]
                err = (out[row, h * D:(h + 1) * D] - want).abs()
                assert (err <= (2.0 ** -11 + ref.half_step(t) + 2.0 ** -20) * want.abs() + 2.0 ** -24).all(), (b, i, h, float(err.max()))
                assert abs(float(lse[row, h]) - first) <= (2 * (D + 8) * 2.0 ** -24) * abs(first)


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("D,G", [(64, 64), (128, 32), (128, 128)])
@pytest.mark.parametrize("t,q,k", [(F16, 1e3, 1e3), (F16, 6e4, 100.0), (F16, 6e4, 4e4), (F16, -6e4, 100.0), (F16, -6e4, 4e4),
                                   (BF16, 1e8, 1.0), (BF16, -1e8, 10.0), (BF16, 1e20, 1e3), (BF16, 1e20, -1e3)])
def test_large_logits(lib, tile, D, G, t, q, k):
    one_hot(lib, tile, t, D, G, q, k)


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("D,G", [(64, 64), (128, 32)])
@pytest.mark.parametrize("q,k", [(6e36, 1.0), (1.2e37, 0.5), (3e38, 1e-3)])
def test_bf16_queries_near_the_end_of_their_range(lib, tile, D, G, q, k):
    one_hot(lib, tile, BF16, D, G, q, k)


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("D,G", [(64, 64), (128, 32)])
@pytest.mark.parametrize("q,k", [(-6e36, 1.0), (-1e32, 1.0), (-1e30, 1.0), (1e28, -1e3)])
def test_logits_far_below_zero(lib, tile, D, G, q, k):
    one_hot(lib, tile, BF16, D, G, q, k)


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("t,q,scale", [(BF16, 1e-37, 1e-25), (BF16, 1e-30, 1e-38), (F16, 1e-6, 1e-38), (F16, 1.0, 1e-38)])
def test_scales_that_leave_nothing_of_the_logits(lib, tile, t, q, scale):
    n0, n1 = TILES[tile]
    s = Setup([(n0, 200), (n1, 90)], 1, 64, 64, 64, t, q_heads=2)
    s.qkv[:, :128] = (s.qkv[:, :128].float() * q).to(t)
    s.fill()
    s.append_model()
    s.device()
    for window in (0, 40):
        out, lse = s.attend(lib, window, scale)
        s.check_attend(out, lse, window, scale, rows=[0, 1, 7, 31, 33, 69])
