"""GPU test of two host threads that fork pools of different sizes at once, each on a stream of its own: what one
asks of the runtime for its launch does not take from the other's."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731


def test_two_threads(lib):
    size = lib.w4a16_kv4_page_bytes(1, 64, 64, 32)
    wrong, ready = [], threading.Barrier(2)

    def work(pages, rows):
        """Only the last `rows` pages are free; each row is a new sequence of one page."""
        try:
            torch.cuda.set_device(0)
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                pool = torch.zeros(pages * size, dtype=torch.uint8, device="cuda")
                pinned = torch.ones(pages, dtype=torch.uint8, device="cuda")
                pinned[pages - rows:] = 0
                table, lens, parent, room = i32([[-1, -1]]), i32([0]), i32([-1] * rows), i32([32] * rows)
                out, held, missing = i32([[9, 9]] * rows), i32([9] * rows), i32([9])
                want = torch.stack([torch.arange(pages - rows, pages, dtype=torch.int32), torch.full((rows,), -1, dtype=torch.int32)], 1)
                stream.synchronize()
                ready.wait()
                for _ in range(200):
                    lib.w4a16_kv4_fork(pool, table, lens, parent, None, room, pinned, out, held, missing, 1, rows, 1, pool.numel(), 1, 64, 64, 32, pages, 2,
                                       stream)
                stream.synchronize()
                if not torch.equal(out.cpu(), want) or missing.item() or held.any():
                    wrong.append((pages, rows))
        except Exception as e:  # noqa: BLE001
            ready.abort()
            wrong.append(repr(e))

    threads = [threading.Thread(target=work, args=a) for a in ((1 << 19, 2048), ((1 << 19) - (1 << 18) + 77, 1500))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not wrong and not any(t.is_alive() for t in threads)
