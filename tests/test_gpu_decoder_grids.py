"""GPU tests of calls with more workgroups than one dimension of a grid takes."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_attention_of_a_long_prompt_among_many_sequences(lib):
    heads, kv, D, page, width, window = 64, 8, 64, 64, 512, 33
    batch, long = 1024, 32768  # a tile is 16 new tokens: 2^24 places for one among these sequences
    g = torch.Generator(device="cuda").manual_seed(3)
    size = 32 * D + 256
    raw = torch.randint(0, 256, (16, kv * page // 32, size), generator=g, device="cuda", dtype=torch.uint8)
    raw[..., 32 * D:] = torch.rand(16, kv * page // 32, 128, generator=g, device="cuda").half().view(torch.uint8)
    raw = raw.contiguous()
    table = torch.randint(0, 16, (batch, width), generator=g, device="cuda", dtype=torch.int32)
    lens = torch.randint(1, 200, (batch,), generator=g, device="cuda", dtype=torch.int32)
    lens[700] = long

    def run(seqs, new, q):
        rows = torch.zeros(len(seqs) + 1, dtype=torch.int32)
        rows[1:] = torch.tensor(new).cumsum(0)
        out = torch.full((int(rows[-1]), heads * D), float("nan"), dtype=torch.float16, device="cuda")
        t = torch.tensor(seqs, device="cuda")
        w = (lens[t].contiguous(), table[t].contiguous())
        lib.w4a16_kv4_attention(q, rows.cuda(), *w, raw, out, None, len(seqs), out.shape[0], max(new), long, heads * D, heads * D,
                                heads, kv, D, D, page, 16, width, window, 0.125, lib.DT_F16)
        torch.cuda.synchronize()
        return out

    new = [1] * batch
    new[700] = long
    q = torch.randn(sum(new), heads * D, generator=g, device="cuda").half()
    out = run(list(range(batch)), new, q)
    assert out.isfinite().all()
    # the same tiles from smaller launches, bit for bit: the prompt alone, and the others among
    # a prompt of 256 (the first of the long one's, at positions that nobody compares)
    assert torch.equal(run([700], [long], q[700:700 + long].contiguous()), out[700:700 + long])
    few = list(new)
    few[700] = 256
    small = run(list(range(batch)), few, torch.cat([q[:956], q[700 + long:]]))
    assert torch.equal(small[:700], out[:700]) and torch.equal(small[956:], out[700 + long:])


def test_norm_of_more_rows_than_a_grid_has_places(lib):
    M, K, part = (1 << 24) + 70, 8, 1 << 19
    g = torch.Generator(device="cuda").manual_seed(4)
    x, gamma = torch.randn(M, K, generator=g, device="cuda").half(), torch.randn(K, generator=g, device="cuda").half()

    def run(x):
        y8, y = torch.empty(x.shape, dtype=torch.uint8, device="cuda"), torch.full_like(x, float("nan"))
        s = torch.full((x.shape[0],), float("nan"), device="cuda")
        lib.w4a8_rmsnorm(x, None, gamma, None, y8, s, y, x.shape[0], K, 1e-5, lib.DT_F16)
        torch.cuda.synchronize()
        return y8, s, y

    whole = run(x)
    for at in (0, part, (1 << 20) - 100, 1 << 20, 5 << 20, M - part):
        for a, b in zip(whole, run(x[at:at + part])):
            assert torch.equal(a[at:at + part], b), at
    assert whole[1].isfinite().all() and whole[2].isfinite().all()
