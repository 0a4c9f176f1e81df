"""GPU tests of prompts and single tokens in one call of attention over the 4-bit cache: every
sequence gets tiles of 128 columns, split between workgroups or not."""
import pytest
import torch

from test_gpu_attend_splits import BF16, F16, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("singles,heads,window", [(32, 8, 0), (32, 8, 5000), (2, 1, 0), (2, 1, 5000)])
def test_long_single_tokens_beside_a_prompt(lib, singles, heads, window, t):
    # 512 tokens of 8 heads and 32 singles make 512 tiles and more: no tile is split
    spread = [(1, 20011)] + [(1, 100 + 37 * i) for i in range(singles - 1)]
    spread.insert(singles // 2, (512, 700))
    c = Case(lib, spread, heads, 8, 64, 64, 64, t, seed=singles, shared=True)
    need = lib.w4a16_kv4_workspace_bytes(len(spread), c.tokens, 512, 20011, heads * 8, heads, 64, window)
    assert (need == 0) == (singles == 32)
    out, lse = c.run(window)
    last = len(spread) - 1
    c.check(out, lse, window, seqs=[0, 1, last] if singles > 2 else [0, last], heads=[0, heads - 1])
    c.check(out, lse, window, seqs=[singles // 2], heads=[heads - 1], rows=[0, 15, 16, 300, 511])
    assert out.isfinite().all() and lse.isfinite().all()


def test_single_tokens_get_what_they_get_alone(lib):
    spread = [(1, 900), (300, 300), (1, 3), (2, 4000), (1, 1)]
    c = Case(lib, spread, 2, 4, 128, 32, 32, F16, seed=9)
    out, lse = c.run()
    c.check(out, lse, seqs=[0, 2, 3, 4])
    c.check(out, lse, seqs=[1], rows=[0, 1, 31, 32, 299])
