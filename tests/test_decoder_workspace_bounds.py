"""How much workspace adapters and attention can need (host code only): the bounds that a stream's
own buffer is made to hold, so that a capture of a smaller shape finds room in it."""
import random

import pytest

w4 = pytest.importorskip("w4a16_mixed_precision_offline_amd")


def test_adapters():
    f, r = w4.w4a16_lora_workspace_bytes, random.Random(1)
    assert f(16, 8192, 8192, 16) > f(17, 8192, 8192, 16)  # which is why one call's need covers nothing
    for _ in range(20000):
        M, rank = int(2 ** r.uniform(0, 21)), 8 * r.randint(1, 16)
        N, K = 8 * int(2 ** r.uniform(0, 14)), 8 * int(2 ** r.uniform(0, 14))
        rp, kr = -(-rank // 16) * 16, 1 if rank <= 32 else 2 if rank <= 64 else 4
        most = max(M, 256) * rp if M <= 512 else max(M, 32768) * rp + -(-M // 64) * (2048 * kr + 64)
        assert 0 < f(M, N, K, rank) <= 4 * most, (M, N, K, rank)


def test_attention():
    f, r = w4.w4a16_kv4_workspace_bytes, random.Random(2)
    assert f(1, 512, 512, 8192, 64, 8, 128) > f(1, 1024, 1024, 8192, 64, 8, 128) == 0
    seen = set()
    for _ in range(20000):
        batch, new, D = int(2 ** r.uniform(0, 11)), int(2 ** r.uniform(0, 12)), r.choice([64, 128])
        kv, ratio = r.choice([1, 2, 5, 8, 32]), r.choice([1, 2, 4, 5, 8, 16])
        tokens = r.randint(new, batch * new)
        cols = 8 if new * ratio <= 8 else 16 if new * ratio <= 128 else 128
        got = f(batch, tokens, new, int(2 ** r.uniform(0, 17)), kv * ratio, kv, D, r.choice([0, 0, 100, 5000]))
        assert got <= 4 * (512 + 1024 * cols * (D + 2)), (batch, new, kv, ratio)
        seen.add((cols, got > 0))
    assert len(seen) == 6
