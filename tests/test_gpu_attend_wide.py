"""GPU tests of the values' ranges in attention's tiles of 128 columns."""
import numpy as np
import pytest
import torch

from test_gpu_decoder_ops import Setup

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
ROWS = [0, 1, 31, 32, 69]


@pytest.mark.parametrize("t,up", [(BF16, 1e20), (BF16, 1e-20), (F16, 2e4), (F16, 1e-4)])
def test_query_range(lib, t, up):
    s = Setup([(70, 100), (17, 60)], 1, 64, 32, 32, t, q_heads=2)
    s.qkv[:, :128] = (s.qkv[:, :128].float().clamp(-3, 3) * up).to(t)
    s.fill()
    s.append_model()
    s.device()
    out, lse = s.attend(lib, 0, 0.125 / up)
    s.check_attend(out, lse, 0, 0.125 / up, rows=ROWS)


@pytest.mark.parametrize("G", [128, 64, 32])
def test_sharp_and_flat_softmax(lib, G):
    s = Setup([(70, 300), (20, 310)], 1, 128, G, 64, F16, q_heads=4)
    s.qkv[:, :512] *= 30                # logits far apart: the reference moves again and again
    s.qkv[0, :128] = 0                  # and all alike
    s.fill()
    s.append_model()
    s.device()
    for scale in (None, 1e-4, 2.0):
        out, lse = s.attend(lib, 0, scale)
        s.check_attend(out, lse, 0, scale, rows=ROWS)


def test_largest_values_saturate(lib):
    s = Setup([(70, 100)], 1, 64, 64, 32, F16, q_heads=2)
    s.fill()
    s.append_model()
    for p in range(100):                # 15 s = 65520 > 65504
        pg = s.table[0, p // 32]
        s.model.s[1, pg, :, p % 32], s.model.m[1, pg, :, p % 32] = 4368, 0
        s.model.c[1, pg, :, p % 32, ::2] = 15
        s.model.write(s.raw, pg, p % 32)
    s.device()
    out, lse = s.attend(lib)
    assert out[:, :128].isfinite().all() and lse.isfinite().all()
    # every value is 65504; p's parts and their sum are off by at most 2^-21 and 2^-17
    assert (out[:, :128:2].double() >= 65504 - 32).all()


@pytest.mark.parametrize("what", [0, 1])
@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("new,G", [(1, 64), (4, 32), (70, 64), (70, 32)])
def test_nan_of_a_seen_token_reaches_those_who_see_it(lib, new, G, t, what):
    """Keys (0) or values (1): the matrix instructions must not lose it."""
    s = Setup([(new, 100), (new, 90)], 1, 64, G, 32, t, q_heads=2)
    s.fill()
    s.append_model()
    at = 50 if new == 70 else 20
    pg = s.table[0, at // 32]
    s.model.m[what, pg, :, at % 32] = np.nan
    s.model.write(s.raw, pg, at % 32)
    s.device()
    out, lse = s.attend(lib)
    first = max(0, at - (100 - new))
    assert out[first:new, :128].isnan().all() and out[new:, :128].isfinite().all()
    assert lse[new:].isfinite().all() and (lse[first:new].isnan().all() if what == 0 else lse[first:new].isfinite().all())
