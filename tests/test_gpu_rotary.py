"""GPU tests of rotary positions against the formula in 64 bits (tests/tree_ref.py)."""
import pytest
import torch

import decoder_ref as ref
import tree_ref as tr

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


class Case:
    def __init__(self, tokens, qh, kh, head, rot, axes, t, neighbours=False, pad=0, seed=0, spread=5000):
        g = torch.Generator().manual_seed(seed)
        self.tokens, self.qh, self.kh, self.head, self.rot, self.axes, self.t, self.neighbours = tokens, qh, kh, head, rot, axes, t, neighbours
        self.width = (qh + 2 * kh) * head + pad
        self.x = torch.randn(tokens, self.width, generator=g).to(t)
        self.pos = torch.randint(-spread, spread, (axes, tokens + 3), generator=g, dtype=torch.int32)
        self.axis = torch.randint(0, axes, (rot // 2,), generator=g, dtype=torch.int32)
        self.freq = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float32) / (rot // 2))

    def parts(self, x):
        q = x[:, :self.qh * self.head]
        return q, x[:, self.qh * self.head:(self.qh + self.kh) * self.head]

    def run(self, w4, in_place=False, stream=None, axis=True, x=None, out=None):
        x = self.x.cuda() if x is None else x
        q, k = self.parts(x)
        if in_place:
            qo, ko, ldo = q, k, (self.width, self.width)
        else:
            if out is None:
                out = [torch.full((self.tokens, n * self.head + 8), float("nan"), dtype=self.t, device="cuda") for n in (self.qh, max(1, self.kh))]
            (qo, ko), ldo = out, (out[0].stride(0), out[1].stride(0))
        w4.w4a16_rotary(q, k if self.kh else None, self.pos.cuda(), self.axis.cuda() if axis else None, self.freq.cuda(), qo, ko if self.kh else None,
                        self.tokens, self.qh, self.kh, self.head, self.rot, self.axes, self.tokens + 3, self.width, self.width, *ldo,
                        w4.ROTARY_NEIGHBOURS if self.neighbours else w4.ROTARY_HALVES, w4.DT_BF16 if self.t == BF16 else w4.DT_F16, stream)
        return x, qo, ko

    def check(self, got, x, heads, axis=None):
        axis = (self.axis if axis is None else axis).long()
        y, tol = tr.rotary(x, heads, self.pos[:, :self.tokens], axis, self.freq, self.neighbours)
        off = (got.double() - y).abs()
        # fp16 below its normal range rounds to steps of 2^-24
        limit = ref.half_step(self.t) * (y.abs() + tol) + tol + 2.0 ** -25
        assert (off <= limit).all(), float((off - limit).max())
        rest = torch.arange(heads * self.head) % self.head >= self.rot
        assert torch.equal(got[:, rest], x[:, rest])


@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("tokens,qh,kh,head,rot,axes", [
    (1, 1, 1, 16, 16, 1), (1, 32, 8, 128, 128, 1), (7, 5, 1, 80, 80, 3), (33, 4, 2, 96, 48, 2), (3, 3, 0, 64, 32, 4), (65, 2, 1, 72, 64, 1),
    (2, 1, 1, 512, 512, 1), (9, 40, 40, 24, 16, 3), (2049, 2, 1, 64, 64, 3), (2051, 1, 2, 88, 16, 1), (130, 64, 8, 128, 64, 1)])
def test_rotary(lib, tokens, qh, kh, head, rot, axes, neighbours, t):
    c = Case(tokens, qh, kh, head, rot, axes, t, neighbours, pad=8 * (head % 3), seed=tokens)
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
    want[:, qh * head:(qh + kh) * head] = ko.cpu()[:, :kh * head]
    assert torch.equal(x.cpu(), want)


@pytest.mark.parametrize("spread", [1 << 20, (1 << 31) - 1])
def test_far_positions(lib, spread):
    c = Case(40, 4, 2, 128, 128, 2, F16, seed=spread % 97, spread=spread)
    c.pos[0, :4] = torch.tensor([0, -2 ** 31, 2 ** 31 - 1, -1], dtype=torch.int32)
    _, qo, ko = c.run(lib)
    q, k = c.parts(c.x)
    c.check(qo.cpu()[:, :512], q, 4)
    c.check(ko.cpu()[:, :256], k, 2)


def test_axes_out_of_range_and_none(lib):
    c = Case(20, 2, 1, 64, 64, 3, BF16, seed=3)
    kept = c.axis.clone()
    c.axis[::3] = -7
    c.axis[1::3] = 1 << 30
    _, qo, _ = c.run(lib)
    c.check(qo.cpu()[:, :128], c.parts(c.x)[0], 2, c.axis.clamp(0, 2))
    assert not torch.equal(kept, c.axis)
    c = Case(20, 2, 1, 64, 64, 1, F16, seed=4)
    _, a, _ = c.run(lib)
    _, b, _ = c.run(lib, axis=False)
    assert torch.equal(a[:, :128], b[:, :128])


def test_backwards_and_edge_values(lib):
    """With -freq the rotation is undone (its transpose, which is its gradient); a pair's NaN and
    infinities stay in that pair."""
    c = Case(64, 4, 4, 64, 64, 1, F16, seed=5)
    x, _, _ = c.run(lib, in_place=True)
    once = x.cpu()
    c.freq = -c.freq
    c.run(lib, in_place=True, x=x)
    # two roundings of values up to |a| + |b|, and the errors of both rotations
    n = c.x.double().abs().view(64, -1, 2, 32)
    limit = (n.sum(2, keepdim=True) * (2 * 2.0 ** -11 + 2 * 2.0 ** -20) + 2.0 ** -23).expand_as(n).reshape(64, -1)[:, :512]
    assert ((x.cpu().double() - c.x.double()).abs()[:, :512] <= limit).all()
    y = once.double()[:, :256]
    assert float((y.square().sum() - c.x.double()[:, :256].square().sum()).abs()) < 64 * 256 * 2.0 ** -9
    c.freq = -c.freq
    c.x[3, 5], c.x[4, 70], c.x[5, 0] = float("nan"), float("inf"), 60000.0
    c.x[5, 32] = 60000.0
    _, qo, _ = c.run(lib)
    got = qo.cpu()[:, :256]
    assert got[3, 5].isnan() and got[3, 37].isnan() and int(got[3].isnan().sum()) == 2
    bad = ~got[4].isfinite()
    assert bad[70] and bad[102] and int(bad.sum()) == 2
    y, _ = tr.rotary(c.x[:, :256], 4, c.pos[:, :64], c.axis.long(), c.freq, False)
    assert torch.equal(got[5].double().isinf(), y[5].abs() >= 65520)  # past fp16's range


def test_gradient_of_the_rotation(lib):
    """d/dx of sum(y w) is the rotation of w by -freq; against differences of the kernel's own output."""
    c = Case(6, 2, 0, 32, 32, 2, F16, seed=6)
    w = torch.randn(6, 64, generator=torch.Generator().manual_seed(7)).half()
    _, y0, _ = c.run(lib)
    back = Case(6, 2, 0, 32, 32, 2, F16, seed=6)
    back.x, back.freq = w.clone(), -c.freq
    _, g, _ = back.run(lib)
    g = g.cpu()[:, :64].double()
    want, _ = tr.rotary(w, 2, c.pos[:, :6], c.axis.long(), -c.freq, False)
    assert ((g - want).abs() <= 2.0 ** -11 * want.abs() + (w.double().abs().max() * 2) * 2.0 ** -20 + 2.0 ** -25).all()
    y0 = y0.cpu()[:, :64].double()
    for i in (0, 5, 16, 40, 63):  # the map is linear: a step of 8 in one channel, within 2^-11 of values up to 13
        step = Case(6, 2, 0, 32, 32, 2, F16, seed=6)
        step.x[:, i] += 8
        dx = (step.x[:, i] - c.x[:, i]).double()
        _, y1, _ = step.run(lib)
        d = ((y1.cpu()[:, :64].double() - y0) * w.double()).sum(1) / dx
        slack = (2 * 2.0 ** -11 * 13 * 2 * w.double().abs().max()) / dx.abs()
        assert ((d - g[:, i]).abs() <= slack + 2.0 ** -11 * g[:, i].abs() + 2.0 ** -10).all()


def test_side_stream_and_graph(lib):
    c = Case(300, 8, 2, 64, 64, 3, BF16, seed=8)
    x = c.x.cuda()
    out = [torch.zeros(300, n * 64, dtype=BF16, device="cuda") for n in (8, 2)]
    pos, axis, freq = c.pos.cuda(), c.axis.cuda(), c.freq.cuda()
    side = torch.cuda.Stream()

    def call(out, stream=None):
        q, k = c.parts(x)
        lib.w4a16_rotary(q, k, pos, axis, freq, *out, 300, 8, 2, 64, 64, 3, 303, c.width, c.width, 512, 128, lib.ROTARY_HALVES, lib.DT_BF16, stream)

    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(out, side)
    for _ in range(3):
        x.normal_()
        pos.random_(0, 100000)
        now = [torch.zeros_like(o) for o in out]
        call(now)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(now, out))


def test_rows_past_4_gib(lib):
    c = Case(24, 2, 1, 64, 64, 1, F16, seed=9)
    ld = (1 << 27) + 8  # 24 rows of 256 MiB
    far = torch.empty(23 * ld + 128, dtype=F16, device="cuda").as_strided((24, 128), (ld, 1))
    far.copy_(c.parts(c.x)[0])
    k = c.parts(c.x)[1].contiguous().cuda()
    args = c.pos.cuda(), None, c.freq.cuda()
    lib.w4a16_rotary(far, k, *args, far, k, 24, 2, 1, 64, 64, 1, 27, ld, 64, ld, 64)
    _, qo, ko = c.run(lib)
    assert torch.equal(far, qo[:, :128]) and torch.equal(k, ko[:, :64])
