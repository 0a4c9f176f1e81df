"""GPU tests of the norm with 8-bit rows over the whole range of its types: rows whose squares or
products with gamma leave fp32 above or below, with eps and without."""
import math

import pytest
import torch

import decoder_ref as ref
from test_gpu_decoder_ops import BF16, F16, rand, run_norm

pytestmark = pytest.mark.gpu
REL = 1e-5  # sums of K squares in chains and a tree, a root, a division, two products in fp32
LEAST = 2.0 ** -126  # of yscale; below it fp32 has no full precision


def check(lib, x, g, eps):
    t = x.dtype
    h, y, s = ref.norm(x, None, g, eps)
    H, Y8, S, Y = run_norm(lib, x, None, g, eps)
    assert torch.equal(H, h) and y.isfinite().all()
    s = s.clamp(min=LEAST)
    assert S.isfinite().all() and ((S.double() - s).abs() <= REL * s).all(), (S, s)
    assert ((Y.double() - y).abs() <= (ref.half_step(t) + REL) * y.abs() + max(LEAST, torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2)).all()
    want = y / S.double()[:, None]
    assert ((Y8 - want).abs() <= (2.0 ** -4 + REL) * want.abs() + 2.0 ** -10).all()


@pytest.mark.parametrize("eps", [0.0, 1e-5])
@pytest.mark.parametrize("K", [8, 4096, 8192, 65536])
def test_rows_of_one_value(lib, K, eps):
    ups = [1e-38, 1e-30, 1e-23, 3e-22, 1e-21, 1e-19, 1e-10, 1e10, 1e18, 1.8e19, 2e19, 1e30, 1e34, 5e36, 1e37, 3e38]
    x = torch.tensor(ups).unsqueeze(1).repeat(1, K).to(BF16)
    check(lib, x, torch.ones(K, dtype=BF16), eps)
    check(lib, x, rand(1, K, t=BF16), eps)


@pytest.mark.parametrize("eps", [0.0, 1e-5])
@pytest.mark.parametrize("K", [64, 2056, 16392, 32776])
def test_random_rows(lib, K, eps):
    x = rand(2, 10, K)
    for i, up in enumerate((1e-37, 1e-30, 1e-22, 1e-20, 1e-3, 1e3, 1e18, 1e30, 1e36, 3e37)):
        x[i] *= up
    x[8, 3] = 1e-30  # far apart in one row
    x[1, 7] = 1e25
    check(lib, x.to(BF16), rand(3, K, t=BF16), eps)


@pytest.mark.parametrize("eps", [0.0, 1e-5])
@pytest.mark.parametrize("up", [1e-36, 1e-20, 1e20, 1e36])
def test_gamma_far_from_one(lib, up, eps):
    # products with h leave fp32, and below 2^-126 * 448 yscale stops
    x = rand(4, 6, 512)
    for i, f in enumerate((1e-36, 1e-20, 1e-10, 1.0, 1e20, 1e36)):
        x[i] *= f
    check(lib, x.to(BF16), (rand(5, 512) * up).to(BF16), eps)


def test_fp16_rows(lib):
    x = rand(6, 5, 1024)
    for i, f in enumerate((1e-7, 1e-5, 1e-2, 1.0, 1.5e4)):
        x[i] *= f
    for eps in (0.0, 1e-5, 1e30):
        check(lib, x.half(), rand(7, 1024, t=F16), eps)


def test_rows_without_a_largest_value(lib):
    x, g = rand(8, 4, 256, t=BF16), torch.ones(256, dtype=BF16)
    x[0] = 0
    for eps in (0.0, 1e-5):
        H, Y8, S, Y = run_norm(lib, x[:1], None, g, eps)
        assert S[0] == 1 and (Y8 == 0).all() and (Y == 0).all()
    H, Y8, S, Y = run_norm(lib, x, None, g, math.inf)  # every y is 0
    assert (S == 1).all() and (Y8 == 0).all() and (Y == 0).all()
    H, Y8, S, Y = run_norm(lib, x, None, torch.zeros_like(g), 1e-5)
    assert (S == 1).all() and (Y8 == 0).all() and (Y == 0).all()
    g[9] = math.inf
    H, Y8, S, Y = run_norm(lib, x[1:], None, g, 1e-5)
    assert (S == 1).all() and Y8[:, 9].isnan().all() and (Y8.nan_to_num() == 0).all()


def test_infinite_and_nan_rows_of_any_magnitude(lib):
    x, g = rand(9, 6, 8192, t=BF16), rand(10, 8192, t=BF16)
    x[1:4] = (x[1:4].float() * 1e37).to(BF16)
    x[0, 100] = x[1, 8000] = math.inf
    x[2, 3] = -math.inf
    x[3, 5] = x[4, 6] = math.nan
    H, Y8, S, Y = run_norm(lib, x, None, g, 1e-5)
    assert (S[:5] == 1).all() and S[5] != 1
    assert Y8[3:5].isnan().all() and torch.equal(Y8[:3].isnan(), x[:3].isinf()) and (Y8[:3].nan_to_num() == 0).all()


@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("K", [8, 4096, 16384, 65536])
def test_rows_of_zeros_among_others(lib, K, t):
    least = torch.tensor([1], dtype=torch.int16).view(t)  # squares to 0 in fp32, for bf16
    x, g = rand(11, 6, K, t=t), rand(12, K, t=t)
    x[0] = x[3] = 0
    x[2] = x[4] = x[5] = -0.0
    x[4, K - 1] = x[5, 0] = least[0]
    for eps in (0.0, 1e-5):
        H, Y8, S, Y = run_norm(lib, x, None, g, eps)
        for m in (0, 2, 3):
            assert S[m] == 1 and (Y8[m] == 0).all() and (Y[m] == 0).all()
        if eps == 0:
            keep = torch.tensor([1, 4, 5])
            _, y, s = ref.norm(x[keep], None, g, eps)
            assert ((S[keep].double() - s).abs() <= REL * s).all()
            assert ((Y[keep].double() - y).abs() <= (ref.half_step(t) + REL) * y.abs() + 2.0 ** -25).all()
