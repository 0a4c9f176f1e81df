"""GPU tests of the adapters' tiles of 64 rows (more than 512 rows), against tests/decoder_ref.py."""
import pytest
import torch

from test_gpu_decoder_ops import check_lora

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("M,N,K,r,mixed", [(513, 256, 520, 16, False), (600, 328, 1032, 64, False), (577, 136, 264, 24, True),
                                           (640, 520, 2048, 128, False), (1030, 72, 8, 40, True)])
def test_tiles_of_many_rows(lib, M, N, K, r, mixed, t):
    g = torch.Generator().manual_seed(M)
    ids = torch.randint(-1, 7, (M,), generator=g, dtype=torch.int32)
    if not mixed:
        ids = ids.sort().values
    check_lora(lib, M, N, K, r, 6, ids, t)


def test_tiles_in_place_strides_and_no_adapter(lib):
    M = 530
    ids = torch.arange(M, dtype=torch.int32) % 3 - 1
    check_lora(lib, M, 264, 512, 16, 2, ids, F16, ldx=520, ldy=280, in_place=True)
    check_lora(lib, M, 264, 512, 16, 2, ids, BF16, ldx=536, ldy=272)
    check_lora(lib, M, 264, 512, 16, 2, torch.full((M,), -1, dtype=torch.int32), F16)
    check_lora(lib, M, 264, 512, 16, 2, torch.full((M,), 2 ** 31 - 1, dtype=torch.int32), F16, in_place=True)


@pytest.mark.parametrize("xs", [1e-6, 3e3])
def test_tiles_small_and_large_intermediates(lib, xs):
    check_lora(lib, 520, 64, 4096, 16, 2, torch.arange(520, dtype=torch.int32) % 2, F16, xs=xs)
