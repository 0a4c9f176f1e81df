"""GPU tests of rotary positions of prompts: more than 512 tokens, where a workgroup has a whole token and a thread
several of its items, with stores past the caches where a head's turned and copied channels fill whole lines."""
import pytest
import torch

from test_gpu_rotary import BF16, F16, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("tokens,qh,kh,head,rot,axes", [
    (513, 40, 8, 128, 128, 3),    # all turned: 384 items a token
    (517, 3, 2, 256, 128, 1),     # half turned, the rest copied, both in whole lines
    (515, 5, 1, 208, 128, 2),     # whole lines turned, 80 channels copied: not past the caches
    (514, 131, 2, 128, 128, 1),   # 1064 items, more than 256 threads have in one pass of four, and no multiple of 256
    (519, 70, 3, 256, 128, 2),    # 1168 items, copied ones among them
    (600, 17, 0, 512, 512, 4)])   # queries alone
def test_rotary_of_prompts(lib, tokens, qh, kh, head, rot, axes, neighbours, t):
    c = Case(tokens, qh, kh, head, rot, axes, t, neighbours, pad=8, seed=tokens + rot)
    x, qo, ko = c.run(lib)
    assert torch.equal(x.cpu(), c.x)
    q, k = c.parts(c.x)
    c.check(qo.cpu()[:, :qh * head], q, qh)
    assert qo.cpu()[:, qh * head:].isnan().all()
    if kh:
        c.check(ko.cpu()[:, :kh * head], k, kh)
        assert ko.cpu()[:, kh * head:].isnan().all()
    x, _, _ = c.run(lib, in_place=True)  # the same bits, and nothing beside q and k
    want = c.x.clone()
    want[:, :qh * head] = qo.cpu()[:, :qh * head]
    if kh:
        want[:, qh * head:(qh + kh) * head] = ko.cpu()[:, :kh * head]
    assert torch.equal(x.cpu(), want)


def test_one_of_two_in_place(lib):
    """Queries in place and keys into rows of their own: what is not turned of the queries is stored over itself."""
    for tokens, head, rot in ((520, 256, 128), (30, 96, 48)):
        c = Case(tokens, 3, 2, head, rot, 1, F16, seed=rot)
        _, qo, ko = c.run(lib)
        x = c.x.cuda()
        q, k = c.parts(x)
        out = torch.full((tokens, 2 * head + 8), float("nan"), dtype=F16, device="cuda")
        lib.w4a16_rotary(q, k, c.pos.cuda(), None, c.freq.cuda(), q, out, tokens, 3, 2, head, rot, 1, tokens + 3, c.width, c.width, c.width, 2 * head + 8,
                         lib.ROTARY_HALVES, lib.DT_F16)
        assert torch.equal(q, qo[:, :3 * head]) and torch.equal(out[:, :2 * head], ko[:, :2 * head]) and torch.equal(k.cpu(), c.parts(c.x)[1])
        assert torch.equal(x[:, 5 * head:].cpu(), c.x[:, 5 * head:]) and out[:, 2 * head:].isnan().all()
