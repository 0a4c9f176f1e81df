"""GPU tests of the workspace of adapters and attention: what one call before a capture covers,
and buffers of the caller's."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu
F16 = torch.float16
HEADS, KV, D, G, PAGE, WIDTH = 16, 2, 64, 64, 64, 64


class Arena:
    """Buffers that every call here fits in."""

    def __init__(self, rows, width=1024):
        g = torch.Generator(device="cuda").manual_seed(1)
        new = lambda *s: torch.randn(*s, generator=g, device="cuda").half()  # noqa: E731
        self.x, self.y, self.base = new(rows, width), new(rows, width), new(rows, width)
        self.A, self.B = new(2, 128 * width), new(2, 128 * width)
        self.ids = torch.randint(-1, 2, (rows,), generator=g, device="cuda", dtype=torch.int32)
        self.scale = torch.ones(2, device="cuda")
        self.q, self.out = new(rows, HEADS * D), new(rows, HEADS * D)
        self.lens = torch.randint(1, PAGE * WIDTH, (64,), generator=g, device="cuda", dtype=torch.int32)
        self.table = torch.randint(0, 8, (64, WIDTH), generator=g, device="cuda", dtype=torch.int32)
        size = 32 * D + 256 * (D // G)  # of a block of 32 tokens of a head
        raw = torch.randint(0, 256, (8, KV * PAGE // 32, size), generator=g, device="cuda", dtype=torch.uint8)
        par = torch.rand(8, KV * PAGE // 32, 256 * (D // G) // 2, generator=g, device="cuda").half()
        raw[..., 32 * D:] = par.view(torch.uint8)
        self.cache = raw.contiguous()

    def lora(self, w4, M, N, K, rank, stream=None):
        w4.w4a16_lora(self.x, self.A, self.B, self.ids, self.scale, self.base, self.y, M, N, K, rank, 2, 1024, 1024, w4.DT_F16, stream)

    def rows(self, batch, new):
        return torch.arange(batch + 1, dtype=torch.int32, device="cuda") * new

    def attend(self, w4, rows, batch, new, max_len, stream=None):
        w4.w4a16_kv4_attention(self.q, rows, self.lens, self.table, self.cache, self.out, None, batch, batch * new, new, max_len,
                               HEADS * D, HEADS * D, HEADS, KV, D, G, PAGE, 8, WIDTH, 0, D ** -0.5, w4.DT_F16, stream)


def captured(calls, side):
    """The calls in one graph, replayed three times beside eager work."""
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for call in calls:
            call(side)
    return graph


@pytest.mark.parametrize("M,rank", [(300, 64), (700, 128), (2048, 16)])
def test_one_call_covers_the_adapters_of_fewer_rows(lib, M, rank):
    a, side, r = Arena(2048), torch.cuda.Stream(), random.Random(M)
    side.wait_stream(torch.cuda.current_stream())
    a.lora(lib, M, 64, 64, rank, side)
    shapes = [(1, 256, 1024, rank), (15, 64, 1024, rank), (16, 64, 1024, rank), (17, 64, 1024, 8)]
    shapes += [(r.randint(1, M), 8 * r.randint(1, 128), 8 * r.randint(1, 128), 8 * r.randint(1, rank // 8)) for _ in range(24)]
    for s in shapes:
        graph = captured([lambda st, s=s: a.lora(lib, *s, st)], side)  # refused if the stream holds too little
        a.lora(lib, *s)
        torch.cuda.synchronize()
        want = a.y.clone()
        for _ in range(3):
            a.y.normal_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(a.y[:s[0], :s[1]], want[:s[0], :s[1]]), s


@pytest.mark.parametrize("batch,new,max_len", [(64, 1, 32), (64, 16, 20), (8, 256, 4096), (1, 2048, 4096)])
def test_one_call_covers_the_attention_of_fewer_tokens(lib, batch, new, max_len):
    a, side, r = Arena(2048), torch.cuda.Stream(), random.Random(new)
    rows = a.rows(batch, new)
    torch.cuda.synchronize()
    a.attend(lib, rows, batch, new, max_len, side)
    shapes = [(1, 1, 4096), (batch, 1, 4096), (1, new, 4096), (1, max(1, new // 2), 4096), (1, max(1, new // 4), 4096)]
    shapes += [(b, r.randint(1, min(new, 2048 // b)), r.randint(1, 4096)) for b in (r.randint(1, 64) for _ in range(16))]
    for s in shapes:
        rows = a.rows(s[0], s[1])
        torch.cuda.synchronize()
        graph = captured([lambda st: a.attend(lib, rows, *s, st)], side)
        a.attend(lib, rows, *s)
        torch.cuda.synchronize()
        want = a.out.clone()
        for _ in range(3):
            a.out.normal_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(a.out[:s[0] * s[1]], want[:s[0] * s[1]]), s


def test_buffers_of_the_callers(lib):
    a, side = Arena(2048), torch.cuda.Stream()
    # (what to run, its workspace): adapters in both tiles, attention in tiles of 8, 16 and 128 columns
    lora = [(m, 1024, 1024, r) for m, r in ((16, 64), (700, 64))]
    attend = [(1, 1, 4096), (2, 9, 4096), (1, 300, 4096)]
    todo = [(lib.w4a16_lora_workspace_bytes(*s), lambda st=None, s=s: a.lora(lib, *s, st), a.y) for s in lora]
    for s in attend:
        need = lib.w4a16_kv4_workspace_bytes(s[0], s[0] * s[1], s[1], s[2], HEADS, KV, D)
        todo.append((need, lambda st=None, s=s, rows=a.rows(s[0], s[1]): a.attend(lib, rows, *s, st), a.out))
    for need, call, out in todo:
        assert need > 0
        out.zero_()
        call()
        torch.cuda.synchronize()
        want = out.clone()
        room = lib.WS_COUNTER_BYTES + need
        buf = torch.zeros(room + 4096, dtype=torch.uint8, device="cuda")
        buf[room:] = 77
        torch.cuda.synchronize()
        lib.w4a16_set_workspace(buf, room, stream=side)
        try:
            for _ in range(2):  # the counters are left at zero
                out.zero_()
                torch.cuda.synchronize()
                call(side)
                side.synchronize()
                assert torch.equal(out, want)
            assert (buf[:lib.WS_COUNTER_BYTES] == 0).all() and (buf[room:] == 77).all()
            lib.w4a16_set_workspace(buf, lib.WS_COUNTER_BYTES + need // 4, stream=side)
            out.fill_(5.0)
            torch.cuda.synchronize()
            with pytest.raises(lib.W4A16Error) as e:
                call(side)
            assert e.value.code == -6
            side.synchronize()
            assert (out == 5.0).all()  # nothing was launched
        finally:
            lib.w4a16_set_workspace(None, 0, stream=side)
