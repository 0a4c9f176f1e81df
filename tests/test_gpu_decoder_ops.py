"""GPU tests of the operators beside the product in a decoder step (norm with 8-bit rows,
adapters, 4-bit cache, attention over it) against tests/decoder_ref.py."""
import math

import numpy as np
import pytest
import torch

import decoder_ref as ref

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


def kind(w4, t):
    return w4.DT_BF16 if t == BF16 else w4.DT_F16


def rand(seed, *shape, scale=1.0, t=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(t)


# ---- norm -------------------------------------------------------------------------------------
def run_norm(w4, x, r, g, eps, in_place=False, both=True):
    M, K = x.shape
    t = x.dtype
    X, R, G = x.cuda(), None if r is None else r.cuda(), g.cuda()
    H = (R if r is not None else X) if in_place else torch.full_like(X, math.nan)
    Y8 = torch.zeros(M, K, dtype=torch.uint8, device="cuda")
    S = torch.full((M,), math.nan, device="cuda")
    Y = torch.full_like(X, math.nan) if both else None
    w4.w4a8_rmsnorm(X, R, G, H, Y8, S, Y, M, K, eps, kind(w4, t))
    return H.cpu(), Y8.cpu().view(torch.float8_e4m3fn).double(), S.cpu(), None if Y is None else Y.cpu()


@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("M,K", [(1, 8), (3, 64), (1, 4096), (5, 2056), (77, 5120), (2, 8192), (3, 8200), (2, 16384),
                                 (1, 16392), (2, 32776), (1, 65536)])
def test_norm(lib, M, K, t):
    x, r, g = rand(1, M, K, t=t), rand(2, M, K, scale=3, t=t), rand(3, K, t=t)
    h, y, s = ref.norm(x, r, g, 1e-5)
    H, Y8, S, Y = run_norm(lib, x, r, g, 1e-5, in_place=M % 2 == 0)
    assert torch.equal(H, h)
    # sums of K squares in chains of at most 64 and a tree: 80 steps of 2^-24, then a square
    # root, a division and two products
    rel = 1e-5
    assert ((S.double() - s).abs() <= rel * s).all()
    assert ((Y.double() - y).abs() <= (ref.half_step(t) + rel) * y.abs() + 2.0 ** -25).all()
    # E4M3: half a step of 2^-3, 2^-10 below the normal range; y / s only moves by rel
    want = y / S.double()[:, None]
    assert ((Y8 - want).abs() <= (2.0 ** -4 + rel) * want.abs() + 2.0 ** -10).all()


def test_norm_without_residual_and_outputs(lib):
    x, g = rand(4, 9, 512, t=F16), rand(5, 512, t=F16)
    _, y, s = ref.norm(x, None, g, 0.0)
    H, Y8, S, Y = run_norm(lib, x, None, g, 0.0, in_place=True, both=False)
    assert torch.equal(H, x) and Y is None
    want = y / S.double()[:, None]
    assert ((Y8 - want).abs() <= (2.0 ** -4 + 1e-5) * want.abs() + 2.0 ** -10).all()
    X, G = x.cuda(), g.cuda()
    Y8b, Sb = torch.zeros(9, 512, dtype=torch.uint8, device="cuda"), torch.zeros(9, device="cuda")
    lib.w4a8_rmsnorm(X, None, G, None, Y8b, Sb, None, 9, 512, 0.0, lib.DT_F16)
    assert torch.equal(Sb.cpu(), S) and torch.equal(Y8b.cpu().view(torch.float8_e4m3fn).double(), Y8)


def test_norm_rows_of_zeros_infinities_nan_and_huge_bf16(lib):
    x = rand(6, 6, 1024, t=BF16)
    x[0] = 0
    x[1, 17] = math.inf
    x[2, 5] = math.nan
    x[3] *= 1e30                       # squares pass the fp32 range
    x[4] = x[4].float().mul(1e-30).to(BF16)
    g = torch.ones(1024, dtype=BF16)
    H, Y8, S, Y = run_norm(lib, x, None, g, 1e-5)
    assert (Y8[0] == 0).all() and S[0] == 1
    assert Y8[1, 17].isnan() and S[1] == 1 and (Y8[1].nan_to_num() == 0).all()
    assert Y8[2].isnan().all() and S[2] == 1
    _, y, s = ref.norm(x[3:], None, g, 1e-5)
    assert ((S[3:].double() - s).abs() <= 1e-5 * s).all()
    assert ((Y.double()[3:] - y).abs() <= (ref.half_step(BF16) + 1e-5) * y.abs()).all()


# ---- adapters ---------------------------------------------------------------------------------
def check_lora(w4, M, N, K, r, adapters, ids, t, ldx=0, ldy=0, in_place=False, xs=1.0, seed=0):
    ldx, ldy = ldx or K, ldy or N
    x = rand(seed + 1, M, ldx, scale=xs, t=t)
    A, B = rand(seed + 2, adapters, r, K, scale=K ** -0.5, t=t), rand(seed + 3, adapters, N, r, scale=0.3, t=t)
    base = rand(seed + 4, M, ldy, t=t)
    scale = 0.5 + rand(seed + 5, adapters).abs()
    X, BASE = x.cuda(), base.cuda()
    Y = BASE if in_place else torch.full_like(BASE, 7.0)
    w4.w4a16_lora(X, A.cuda(), B.cuda(), ids.cuda(), scale.cuda(), BASE, Y, M, N, K, r, adapters, ldx, ldy, kind(w4, t))
    got = Y.cpu()
    if ldy > N:  # what lies between the rows stays
        assert torch.equal(got[:, N:], base[:, N:] if in_place else torch.full_like(got[:, N:], 7.0))
    want, slack = ref.lora(x[:, :K], A, B, ids, scale, base[:, :N])
    err = (got[:, :N].double() - want).abs()
    assert (err <= ref.half_step(t) * want.abs() + slack * (1 + ref.half_step(t)) + 2.0 ** -25).all(), (err - slack).max()
    none = (ids < 0) | (ids >= adapters)
    assert torch.equal(got[none, :N], base[none, :N])


@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("M,N,K,r,adapters", [
    (1, 8, 8, 8, 1), (1, 256, 512, 16, 3), (5, 1000, 264, 24, 2), (16, 320, 1024, 8, 16), (17, 72, 1032, 32, 4),
    (48, 528, 2048, 16, 64), (64, 64, 512, 64, 5), (33, 264, 640, 128, 3)])
def test_lora_few_rows(lib, M, N, K, r, adapters, t):
    g = torch.Generator().manual_seed(M)
    ids = torch.randint(-1, adapters + 1, (M,), generator=g, dtype=torch.int32)
    ids[0] = 0
    check_lora(lib, M, N, K, r, adapters, ids, t)


@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("M,N,K,r,mixed", [(65, 256, 512, 16, False), (200, 328, 1032, 64, False), (130, 136, 264, 24, True),
                                           (300, 520, 512, 128, False), (129, 64, 128, 40, True)])
def test_lora_many_rows(lib, M, N, K, r, mixed, t):
    g = torch.Generator().manual_seed(M)
    ids = torch.randint(-1, 7, (M,), generator=g, dtype=torch.int32)
    if not mixed:
        ids = ids.sort().values
    check_lora(lib, M, N, K, r, 6, ids, t)


@pytest.mark.parametrize("M", [3, 100])
def test_lora_in_place_strides_and_no_adapter(lib, M):
    ids = torch.arange(M, dtype=torch.int32) % 3 - 1
    check_lora(lib, M, 264, 512, 16, 2, ids, F16, ldx=520, ldy=280, in_place=True)
    check_lora(lib, M, 264, 512, 16, 2, ids, BF16, ldx=536, ldy=272)
    check_lora(lib, M, 264, 512, 16, 2, torch.full((M,), -1, dtype=torch.int32), F16)
    check_lora(lib, M, 264, 512, 16, 2, torch.full((M,), 2 ** 31 - 1, dtype=torch.int32), F16, in_place=True)


@pytest.mark.parametrize("xs", [1e-6, 3e3])
def test_lora_small_and_large_intermediates(lib, xs):
    # T far below fp16's range, and above it
    check_lora(lib, 4, 64, 4096, 16, 2, torch.tensor([0, 1, 1, 0], dtype=torch.int32), F16, xs=xs)


# ---- cache ------------------------------------------------------------------------------------
class Setup:
    """Sequences of given (new, length), pages in random order, tokens put in the model."""

    def __init__(self, spread, heads, D, G, page, t, q_heads=0, seed=0, loud=1.0, extra=2):
        g = np.random.default_rng(seed)
        self.spread, self.heads, self.D, self.G, self.page, self.t = spread, heads, D, G, page, t
        self.q_heads = q_heads
        used = [max(0, -(-L // page)) for _, L in spread]
        self.pages = sum(used) + extra
        order = g.permutation(self.pages)
        self.width = max(used + [1]) + 1
        self.table = np.full((len(spread), self.width), -1, np.int32)
        at = 0
        for b, u in enumerate(used):
            self.table[b, :u] = order[at:at + u]
            at += u
        self.rows = np.concatenate([[0], np.cumsum([n for n, _ in spread])]).astype(np.int32)
        self.lens = np.array([L for _, L in spread], np.int32)
        self.tokens = max(1, int(self.rows[-1]))
        self.max_new = max([n for n, _ in spread] + [1])
        self.max_len = max([L for _, L in spread] + [1])
        self.model = ref.Cache(self.pages, heads, D, G, page)
        self.raw = g.integers(0, 256, (self.pages, heads * (page // 32) * self.model.block_bytes()), dtype=np.uint8)
        self.raw[:, -64:] = 255  # what was never written may be NaN
        cols = (q_heads + 2 * heads) * D
        self.qkv = torch.from_numpy(g.standard_normal((self.tokens, cols)).astype(np.float32)).to(t)
        self.qkv[:, q_heads * D:(q_heads + heads) * D] *= loud
        self.g = g

    def fill(self):
        """Held tokens, straight into the model and the raw bytes."""
        for b, (n, L) in enumerate(self.spread):
            for p in range(max(0, L - n)):
                k, v = (torch.from_numpy(self.g.standard_normal((self.heads, self.D)).astype(np.float32)).to(self.t).float().numpy()
                        for _ in range(2))
                pg = self.table[b, p // self.page]
                self.model.put(pg, p % self.page, k, v)
                self.model.write(self.raw, pg, p % self.page)

    def append_model(self):
        D, h, qh = self.D, self.heads, self.q_heads
        f = self.qkv.float().numpy()
        for b, (n, L) in enumerate(self.spread):
            for i in range(n):
                p = L - n + i
                if p < 0 or p // self.page >= self.width or not 0 <= self.table[b, p // self.page] < self.pages:
                    continue
                x = f[self.rows[b] + i]
                k = x[qh * D:(qh + h) * D].reshape(h, D)
                v = x[(qh + h) * D:].reshape(h, D)
                pg = self.table[b, p // self.page]
                self.model.put(pg, p % self.page, k, v)
                self.model.write(self.raw, pg, p % self.page)

    def device(self):
        self.d = {n: torch.from_numpy(np.ascontiguousarray(getattr(self, n))).cuda() for n in ("rows", "lens", "table", "raw")}
        self.d["qkv"] = self.qkv.cuda()

    def parts(self):
        D, h, qh = self.D, self.heads, self.q_heads
        return self.d["qkv"].split([qh * D, h * D, h * D], 1)

    def layout(self):
        return self.heads, self.D, self.G, self.page, self.pages, self.width

    def append(self, w4, stream=None):
        _, k, v = self.parts()
        ld = self.qkv.shape[1]
        w4.w4a16_kv4_append(k, v, self.d["rows"], self.d["lens"], self.d["table"], self.d["raw"], len(self.spread), self.tokens,
                            self.max_new, ld, ld, *self.layout(), kind(w4, self.t), stream)

    def gather(self, w4):
        hd = self.heads * self.D
        k, v = (torch.full((self.tokens, hd + 8), math.nan, dtype=self.t, device="cuda") for _ in range(2))
        w4.w4a16_kv4_gather(self.d["raw"], self.d["rows"], self.d["lens"], self.d["table"], k, v, len(self.spread), self.tokens,
                            self.max_new, hd + 8, hd + 8, *self.layout(), kind(w4, self.t))
        return k.cpu(), v.cpu()

    def attend(self, w4, window=0, scale=None, stream=None, out=None, lse=None):
        q = self.parts()[0]
        w = self.q_heads * self.D
        if out is None:
            out = torch.full((self.tokens, w + 8), math.nan, dtype=self.t, device="cuda")
            lse = torch.full((self.tokens, self.q_heads), math.nan, device="cuda")
        w4.w4a16_kv4_attention(q, self.d["rows"], self.d["lens"], self.d["table"], self.d["raw"], out, lse, len(self.spread),
                               self.tokens, self.max_new, self.max_len, self.qkv.shape[1], w + 8, self.q_heads, *self.layout(),
                               window, scale or self.D ** -0.5, kind(w4, self.t), stream)
        return out, lse

    def check_attend(self, out, lse, window=0, scale=None, rows=None):
        scale = scale or self.D ** -0.5
        out, lse = out.cpu(), lse.cpu().double()
        ratio = self.q_heads // self.heads
        assert out[:, self.q_heads * self.D:].isnan().all()
        step = ref.half_step(self.t)
        for b, (n, L) in enumerate(self.spread):
            vals = np.full((max(L, 0), 2, self.heads, self.D), np.nan)
            have = np.zeros(max(L, 0), bool)
            for p in range(max(L, 0)):
                pg = self.table[b, p // self.page] if p // self.page < self.width else -1
                if 0 <= pg < self.pages:
                    vals[p] = self.model.values(pg, p % self.page)
                    have[p] = True
            vals = torch.from_numpy(vals)
            for i in range(n) if rows is None else [i for i in rows if i < n]:
                row, at = self.rows[b] + i, L - n + i
                pos = np.arange(max(L, 0))
                seen = torch.from_numpy(have & (pos <= at) & ((pos > at - window) if window else True))
                for h in range(self.q_heads):
                    q = self.qkv[row, h * self.D:(h + 1) * self.D].double()
                    k, v = vals[:, 0, h // ratio], vals[:, 1, h // ratio]
                    o, l, otol, ltol = ref.attend(q, k, v, seen, scale, self.t)
                    got = out[row, h * self.D:(h + 1) * self.D].double()
                    err = (got - o).abs()
                    assert (err <= step * o.abs() + otol * (1 + step) + 2.0 ** -25).all(), (b, i, h, float((err - otol).max()))
                    if l == -math.inf:
                        assert lse[row, h] == -math.inf
                    else:
                        assert abs(float(lse[row, h]) - l) <= ltol, (b, i, h, float(lse[row, h]) - l, ltol)


@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("D,G,heads,page", [(128, 32, 2, 32), (128, 64, 1, 64), (128, 128, 3, 96), (64, 32, 2, 64), (64, 64, 1, 128)])
def test_append_and_gather_bytes(lib, D, G, heads, page, t):
    s = Setup([(1, 1), (1, 33), (7, 50), (70, 131), (0, 40), (32, 64), (5, 3)], heads, D, G, page, t, seed=D + G, loud=5.0)
    s.fill()
    s.device()
    s.append(lib)
    s.append_model()
    assert np.array_equal(s.d["raw"].cpu().numpy(), s.raw)
    k, v = s.gather(lib)
    hd = heads * D
    assert k[:, hd:].isnan().all() and v[:, hd:].isnan().all()
    for b, (n, L) in enumerate(s.spread):
        for i in range(n):
            p = L - n + i
            if p < 0:
                assert k[s.rows[b] + i].isnan().all()
                continue
            want = torch.from_numpy(s.model.values(s.table[b, p // page], p % page)).to(t).view(2, hd)
            assert torch.equal(k[s.rows[b] + i, :hd], want[0]) and torch.equal(v[s.rows[b] + i, :hd], want[1])


def test_append_edge_values_and_missing_pages(lib):
    s = Setup([(40, 70), (3, 35)], 1, 64, 32, 32, BF16)
    x = s.qkv
    x[0] = 0.0                          # s = 0
    x[1] = 1e30                         # clamped, constant
    x[2, ::2] = -1e30
    x[3, 5] = math.nan
    x[4, 70] = math.inf
    x[5] *= 1e-8                        # s and m below fp16's range
    x[6] = x[6].float().mul(1e-4).to(BF16)
    s.table[0, 1] = -1                  # positions 32 .. 63 have no page
    s.table[1, 1] = s.pages             # nor has position 32 and on of the second
    s.device()
    s.append(lib)
    s.append_model()
    got, want = s.d["raw"].cpu().numpy(), s.raw
    model = s.model
    # a NaN has many bit patterns; its places hold one, everything else is equal
    n = (got != want).sum()
    k, v = s.gather(lib)
    assert n <= 4 * 2
    for b, (cnt, L) in enumerate(s.spread):
        for i in range(cnt):
            p, row = L - cnt + i, s.rows[b] + i
            pg = s.table[b, p // 32]
            if not 0 <= pg < s.pages:
                assert (k[row, :64] == 0).all() and (v[row, :64] == 0).all()
                continue
            w = torch.from_numpy(model.values(pg, p % 32)).to(BF16).view(2, 64)
            for a, c in ((k, w[0]), (v, w[1])):
                assert torch.equal(a[row, :64].isnan(), c.isnan())
                assert torch.equal(a[row, :64].nan_to_num(), c.nan_to_num())


def test_cache_places_past_4_gib(lib):
    heads, D, G, page = 32, 128, 32, 256
    size = lib.w4a16_kv4_page_bytes(heads, D, G, page)
    pages = (1 << 32) // size + 40
    s = Setup([(2, 300)], heads, D, G, page, F16, q_heads=32)
    cache = torch.zeros(pages, size, dtype=torch.uint8, device="cuda")
    ids = [pages - 1, pages - 7]
    s.device()
    small = s.d["raw"]
    s.append(lib)
    cache[ids] = small[[int(s.table[0, 0]), int(s.table[0, 1])]]
    a, la = s.attend(lib)
    s.d["raw"], s.pages = cache, pages
    s.d["table"] = torch.tensor([ids + [-1]], dtype=torch.int32, device="cuda")
    s.append(lib)
    b, lb = s.attend(lib)
    # the held places are random bytes: the same bits give the same results wherever they lie
    assert torch.equal(a.view(torch.int16), b.view(torch.int16)) and torch.equal(la.view(torch.int32), lb.view(torch.int32))


# ---- attention ----------------------------------------------------------------------------------
@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("D,G,heads,ratio,page,window", [
    (128, 128, 2, 8, 64, 0), (128, 64, 1, 4, 32, 0), (128, 32, 2, 1, 96, 0), (64, 64, 1, 16, 64, 0), (64, 32, 3, 5, 32, 0),
    (128, 64, 1, 8, 64, 20), (64, 32, 1, 2, 32, 1), (128, 128, 1, 3, 32, 70)])
def test_attend_single_tokens(lib, D, G, heads, ratio, page, window, t):
    s = Setup([(1, 1), (1, 2), (1, 32), (1, 33), (1, 200), (0, 5), (1, 700)], heads, D, G, page, t, q_heads=heads * ratio,
              seed=ratio)
    s.fill()
    s.append_model()
    s.device()
    out, lse = s.attend(lib, window)
    s.check_attend(out, lse, window)


@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("D,G,heads,ratio,page,window", [
    (128, 128, 1, 8, 64, 0), (128, 64, 2, 4, 32, 0), (128, 32, 1, 1, 64, 0), (64, 64, 2, 5, 96, 0), (64, 32, 1, 16, 32, 0),
    (128, 128, 1, 8, 32, 37), (64, 64, 1, 2, 32, 130), (128, 32, 1, 3, 64, 3)])
def test_attend_many_tokens(lib, D, G, heads, ratio, page, window, t):
    s = Setup([(3, 3), (70, 70), (33, 250), (129, 300), (2, 65), (1, 90), (0, 0), (16, 48)], heads, D, G, page, t,
              q_heads=heads * ratio, seed=D + ratio)
    s.fill()
    s.append_model()
    s.device()
    out, lse = s.attend(lib, window)
    s.check_attend(out, lse, window, rows=[0, 1, 2, 15, 16, 31, 32, 33, 63, 64, 69, 100, 127, 128])


def test_attend_missing_pages_and_empty_rows(lib):
    s = Setup([(40, 96), (2, 64), (5, 3)], 1, 128, 64, 32, F16, q_heads=8)
    s.fill()
    s.append_model()
    s.table[0, 0] = -1
    s.table[0, 2] = 2 ** 31 - 1
    s.table[1, :2] = -1                 # nothing to see at all
    s.device()
    out, lse = s.attend(lib)
    s.check_attend(out, lse)
    assert (out[40:42, :1024] == 0).all() and (lse[40:42] == -math.inf).all()
    out, lse = s.attend(lib, 8)
    s.check_attend(out, lse, 8)


def test_attend_nan_and_infinity_in_places_nobody_sees(lib):
    for new in (1, 64):
        s = Setup([(new, 75 + new)], 2, 128, 32, 64, F16, q_heads=8)
        s.fill()
        s.append_model()
        for p in list(range(0, 40)) + list(range(75 + new, 192)):  # before the window, behind the end
            pg, t = s.table[0, p // 64], p % 64
            if pg < 0:
                continue
            s.model.s[:, pg, :, t] = np.inf if p % 2 else np.nan
            s.model.m[:, pg, :, t] = np.nan if p % 3 else -np.inf
            s.model.write(s.raw, pg, t)
        s.device()
        window = 75 + 1 - 40
        out, lse = s.attend(lib, window)
        s.check_attend(out, lse, window)


def test_attend_sharp_and_flat_softmax(lib):
    s = Setup([(1, 300), (20, 310)], 1, 128, 128, 64, F16, q_heads=4)
    s.qkv[:, :512] *= 30                # logits far apart: the reference moves again and again
    s.qkv[0, :128] = 0                  # and all alike
    s.fill()
    s.append_model()
    s.device()
    for scale in (None, 1e-4, 2.0):
        out, lse = s.attend(lib, 0, scale)
        s.check_attend(out, lse, 0, scale)


@pytest.mark.parametrize("t,up", [(BF16, 1e20), (BF16, 1e-20), (F16, 2e4), (F16, 1e-4)])
def test_attend_query_range(lib, t, up):
    s = Setup([(1, 100), (17, 60)], 1, 64, 32, 32, t, q_heads=2)
    s.qkv[:, :128] = (s.qkv[:, :128].float().clamp(-3, 3) * up).to(t)
    s.fill()
    s.append_model()
    s.device()
    out, lse = s.attend(lib, 0, 0.125 / up)
    s.check_attend(out, lse, 0, 0.125 / up)


def test_attend_largest_values_saturate(lib):
    s = Setup([(1, 40), (20, 40)], 1, 64, 64, 32, F16, q_heads=2)
    s.fill()
    s.append_model()
    for p in range(40):                 # 15 s = 65520 > 65504
        for b in (0, 1):
            pg = s.table[b, p // 32]
            s.model.s[1, pg, :, p % 32], s.model.m[1, pg, :, p % 32] = 4368, 0
            s.model.c[1, pg, :, p % 32, ::2] = 15
            s.model.write(s.raw, pg, p % 32)
    s.device()
    out, lse = s.attend(lib)
    assert out[:, :128].isfinite().all()
    assert (out[:, :128:2].double() == 65504).all()


def test_attend_rows_beyond_the_bounds_are_left_alone(lib):
    s = Setup([(4, 40), (4, 30)], 1, 64, 64, 32, F16, q_heads=1)
    s.fill()
    s.append_model()
    s.device()
    s.d["rows"] = torch.tensor([-5, 4, 2 ** 31 - 1], dtype=torch.int32, device="cuda")  # brought to 0, 4, 8
    out, lse = s.attend(lib)
    s.check_attend(out, lse)
    s.d["rows"] = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    s.max_new = 3                       # the fourth of each is left alone, the others keep their positions
    out, lse = s.attend(lib)
    assert out[[3, 7], :64].isnan().all() and lse[[3, 7]].isnan().all()
    out[[3, 7], :64] = 0
    full, flse = s.d, None
    s.max_new = 4
    again, alse = s.attend(lib)
    keep = [0, 1, 2, 4, 5, 6]
    assert torch.equal(out[keep, :64], again[keep, :64]) and torch.equal(lse[keep], alse[keep])
    s.max_len = 1                       # lens above max_len: slower, but right
    out, lse = s.attend(lib)
    s.check_attend(out, lse)


def test_attend_reproducible_on_a_side_stream_and_in_a_graph(lib):
    s = Setup([(1, 900), (1, 1500), (1, 3)], 2, 128, 64, 64, F16, q_heads=16)
    s.device()
    s.append(lib)
    s.d["raw"][:] = torch.randint(0, 60, s.d["raw"].shape, dtype=torch.uint8, device="cuda")
    out0, lse0 = s.attend(lib)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        out1, lse1 = s.attend(lib, stream=side)
        x = torch.randn(3, 512, device="cuda").half()
        A, B = torch.randn(2, 16, 512, device="cuda").half(), torch.randn(2, 64, 16, device="cuda").half()
        ids, sc = torch.tensor([1, -1, 0], dtype=torch.int32, device="cuda"), torch.ones(2, device="cuda")
        base, y0 = torch.randn(3, 64, device="cuda").half(), torch.empty(3, 64, device="cuda").half()
        lib.w4a16_lora(x, A, B, ids, sc, base, y0, 3, 64, 512, 16, 2, 512, 64, lib.DT_F16, side)
    side.synchronize()
    assert torch.equal(out0[:, :2048], out1[:, :2048]) and torch.equal(lse0, lse1)
    graph = torch.cuda.CUDAGraph()
    out2, lse2, y1 = torch.zeros_like(out0), torch.zeros_like(lse0), torch.zeros_like(y0)
    with torch.cuda.graph(graph, stream=side):
        s.append(lib, side)
        s.attend(lib, stream=side, out=out2, lse=lse2)
        lib.w4a16_lora(x, A, B, ids, sc, base, y1, 3, 64, 512, 16, 2, 512, 64, lib.DT_F16, side)
    for i in range(3):
        s.d["qkv"].normal_()
        s.append(lib)
        out0, lse0 = s.attend(lib)
        x.normal_()
        lib.w4a16_lora(x, A, B, ids, sc, base, y0, 3, 64, 512, 16, 2, 512, 64)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out0[:, :2048], out2[:, :2048]) and torch.equal(lse0, lse2) and torch.equal(y0, y1)
