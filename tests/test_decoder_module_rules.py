"""What the decoder classes (decoder.py) keep and refuse when the model around them is cast,
moved, saved or trained: host code only, nothing here reaches a kernel."""
import pytest
import torch

pytest.importorskip("w4a16_mixed_precision_offline_amd")
from w4a16_mixed_precision_offline_amd.decoder import Adapters, AttentionBlock, Batch, Kv4Cache  # noqa: E402
from w4a16_mixed_precision_offline_amd.layer import W4A16Linear  # noqa: E402


def half(*shape):
    return torch.zeros(shape, dtype=torch.float16)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def adapters():
    return Adapters(half(2, 8, 64), half(2, 64, 8), torch.tensor([1 / 3, 3e5]))


def block(cache=None):
    return AttentionBlock(half(256), W4A16Linear(256, 512, device="cpu"), W4A16Linear(256, 256, device="cpu"),
                          cache or Kv4Cache(4, 2, 64, 64, 32, device="cpu"), 4)


@pytest.mark.parametrize("cast", [lambda m: m.half(), lambda m: m.bfloat16(), lambda m: m.to(torch.float16), lambda m: m.double(),
                                  lambda m: torch.nn.ModuleList([m]).half()[0]])
def test_a_cast_leaves_the_adapters_scale_as_it_is(cast):
    # the kernel reads it as fp32, and 3e5 has no fp16
    a = adapters()
    cast(a)
    assert a.scale.dtype == torch.float32 and torch.equal(a.scale, torch.tensor([1 / 3, 3e5]))


def test_adapters_refuse_weights_of_another_type():
    x, y, ids = half(3, 64), half(3, 64), i32(3)
    a = adapters()
    a.scale = a.scale.half()
    with pytest.raises(TypeError, match="scale"):
        a(x, y, ids)
    a = adapters()
    a.B = a.B.bfloat16()
    with pytest.raises(TypeError):
        a(x, y, ids)
    a = adapters()
    a.float()
    with pytest.raises(TypeError):
        a(x, y, ids)
    a = adapters()
    a.A = half(2, 64, 8).transpose(1, 2)  # the kernel reads [adapters][rank][in]
    with pytest.raises(ValueError):
        a(x, y, ids)


@pytest.mark.parametrize("cast", [torch.bfloat16, torch.float32])
def test_block_refuses_a_gamma_of_another_type(cast):
    b = block()
    b.to(cast)
    with pytest.raises(TypeError, match="gamma"):
        b(half(2, 256), None, Batch(i32(3), i32(2), i32(2, 2), 1, 32))


def test_host_tensors_are_refused():
    # their addresses would go to a kernel
    cache, b = Kv4Cache(4, 2, 64, 64, 32, device="cpu"), Batch(i32(3), i32(2), i32(2, 2), 1, 32)
    for call in (lambda: cache.append(half(2, 128), half(2, 128), b), lambda: cache.gather(half(2, 128), half(2, 128), b),
                 lambda: cache.attend(half(2, 256), b, 4), lambda: adapters()(half(3, 64), half(3, 64), i32(3)),
                 lambda: block()(half(2, 256), None, b)):
        with pytest.raises(ValueError, match="device"):
            call()


def test_tensors_of_one_call_lie_on_the_current_gpu(monkeypatch):
    from types import SimpleNamespace
    from w4a16_mixed_precision_offline_amd import decoder
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    on = [SimpleNamespace(device=torch.device(d)) for d in ("cuda:1", "cuda:1", "cuda:0", "cpu")]
    decoder._one_gpu(on[0], on[1], None, on[0])
    for odd in (on[2], on[3]):
        with pytest.raises(ValueError, match="device"):
            decoder._one_gpu(odd, on[0])
        with pytest.raises(ValueError, match="device"):
            decoder._one_gpu(on[0], None, on[1], odd)


def test_the_cache_is_no_part_of_a_checkpoint():
    b = block()
    state = b.state_dict()
    assert "gamma" in state and not any(n.startswith("cache") for n in state)
    other = block(Kv4Cache(9, 2, 64, 64, 32, device="cpu"))  # another number of pages
    other.load_state_dict(state)
    assert dict(other.named_buffers())["cache.data"].shape[0] == 9
    # one that was saved with the pages in it loads, and leaves them alone
    old = {**state, "cache.data": torch.ones(4, 4, dtype=torch.uint8)}
    before = other.cache.data.clone()
    other.load_state_dict(old)
    assert torch.equal(other.cache.data, before)
    other.cache.load_state_dict({"data": old["cache.data"]})
    with pytest.raises(RuntimeError):
        other.load_state_dict({**state, "cache.pages": torch.ones(1)})


def test_rows_of_no_sequence_attend_to_nothing(monkeypatch):
    # the kernel leaves them alone: what the caller gets must not be memory of earlier tensors
    from w4a16_mixed_precision_offline_amd import decoder
    monkeypatch.setattr(decoder, "_one_gpu", lambda *x: None)
    monkeypatch.setattr(decoder, "w4a16_kv4_attention", lambda *x: None)
    torch.use_deterministic_algorithms(True)  # torch.empty gives NaN
    try:
        cache = Kv4Cache(4, 2, 64, 64, 32, device="cpu")
        out = cache.attend(half(5, 256), Batch(i32(3), i32(2), i32(2, 2), 1, 32), 4)
    finally:
        torch.use_deterministic_algorithms(False)
    assert out.shape == (5, 256) and (out == 0).all()


def test_adapters_refuse_to_write_behind_autograd():
    # the kernel writes y in place where no gradient sees it
    a, y = adapters(), half(3, 64).requires_grad_()
    with pytest.raises(ValueError, match="gradient"):
        a(half(3, 64), y, i32(3))
    with torch.no_grad(), pytest.raises(ValueError, match="device"):  # past that check
        a(half(3, 64), y, i32(3))
    with pytest.raises(ValueError, match="device"):  # no gradient reaches x, as with the linear layers
        a(half(3, 64).requires_grad_(), half(3, 64), i32(3))
