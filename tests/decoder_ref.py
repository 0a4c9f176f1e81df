"""Plain definitions, in 64 bits on the CPU, of the operators beside the product in a decoder
step: the norm with 8-bit rows, the adapters, the 4-bit cache (byte for byte) and the
attention over it.  Written from the formulas in include/w4a16.h; shares no code with the
library."""
import math

import numpy as np
import torch

NIB = [e // 2 + 4 * (e % 2) for e in range(8)]


def half_step(t):
    return torch.finfo(t).eps / 2


# ---- norm ---------------------------------------------------------------------------------
def norm(x, r, g, eps):
    """h (in x's type), y and yscale in fp64."""
    h = x if r is None else (x.float() + r.float()).to(x.dtype)
    f = h.double()
    y = f / torch.sqrt(f.square().mean(1, keepdim=True) + eps) * g.double()
    s = y.abs().amax(1) / 448
    return h, y, torch.where(s > 0, s, 1.0)


# ---- adapters -----------------------------------------------------------------------------
def lora(x, A, B, ids, scale, base):
    """Y in fp64 and the largest error a result may have beside its own rounding."""
    y, slack = base.double(), torch.zeros(base.shape, dtype=torch.float64)
    K, r = x.shape[1], A.shape[1]
    split = 2.0 ** -17 if x.dtype == torch.bfloat16 else 2.0 ** -21  # T as two 16-bit numbers
    for m, a in enumerate(ids.tolist()):
        if not 0 <= a < A.shape[0]:
            continue
        t = A[a].double() @ x[m].double()
        tabs = A[a].double().abs() @ x[m].double().abs()
        s = float(scale[a])
        y[m] += s * (B[a].double() @ t)
        # fp32 sums of K and then r products; one fused multiply-add into the base
        slack[m] = abs(s) * (B[a].double().abs() @ (K * 2.0 ** -24 * tabs + (split + (2 * r + 4) * 2.0 ** -24) * t.abs()))
        slack[m] += 2.0 ** -23 * y[m].abs()
    return y, slack


# ---- 4-bit cache ---------------------------------------------------------------------------
def quantize(x, group):
    """x fp32 numpy [..., D] -> codes uint8, s and m fp16 [..., D/G]."""
    x = np.asarray(x, np.float32)
    v = np.clip(x, -65504, 65504).reshape(*x.shape[:-1], -1, group)
    lo, hi = v.min(-1), v.max(-1)  # NaN where the group has one
    m, s = lo.astype(np.float16), ((hi - lo) / np.float32(15)).astype(np.float16)
    sf = s.astype(np.float32)[..., None]
    with np.errstate(invalid="ignore", divide="ignore"):
        c = np.rint((v - m.astype(np.float32)[..., None]) / sf)
    c = np.where(sf > 0, np.clip(c, 0, 15), 0)
    return np.nan_to_num(c).astype(np.uint8).reshape(x.shape), s, m


class Cache:
    """One sequence-independent model of the pages: codes and parameters by
    (page, kv head, token in page), for keys (0) and values (1)."""

    def __init__(self, pages, heads, D, G, page):
        self.pages, self.heads, self.D, self.G, self.page = pages, heads, D, G, page
        shape = (2, pages, heads, page)
        self.c = np.zeros(shape + (D,), np.uint8)
        self.s = np.zeros(shape + (D // G,), np.float16)
        self.m = np.zeros(shape + (D // G,), np.float16)

    def put(self, page, t, k, v):
        """k, v [heads, D] fp32 of the token at place t of the page."""
        for i, x in enumerate((k, v)):
            self.c[i, page, :, t], self.s[i, page, :, t], self.m[i, page, :, t] = quantize(x, self.G)

    def values(self, page, t):
        """[2, heads, D] in fp64."""
        s = np.repeat(self.s[:, page, :, t].astype(np.float64), self.G, -1)
        m = np.repeat(self.m[:, page, :, t].astype(np.float64), self.G, -1)
        with np.errstate(invalid="ignore"):
            return m + s * self.c[:, page, :, t]

    def block_bytes(self):
        return 32 * self.D + 256 * (self.D // self.G)

    def code_place(self, is_v, t, d):
        """(byte in the block, shift) of token t (0..31), channel d."""
        if is_v:
            e = t // 16 * 4 + t % 4
            word = (d // 64 * 64 + t // 4 % 4 * 16 + d % 16) * 4 + d % 64 // 16
            base = 16 * self.D
        else:
            e = d % 8
            word = (t // 16 * 64 + d % 32 // 8 * 16 + t % 16) * (self.D // 32) + d // 32
            base = 0
        return base + 4 * word + NIB[e] // 2, 4 * (NIB[e] % 2)

    def param_place(self, is_v, t, q, which):
        n = self.D // self.G
        return 32 * self.D + 128 * n * is_v + 2 * (q * 64 + which * 32 + 8 * (t // 4 % 4) + 4 * (t // 16) + t % 4)

    def write(self, raw, page, t):
        """Put token t of the page into raw [pages, page bytes]."""
        size = self.block_bytes()
        n = self.D // self.G
        for h in range(self.heads):
            at = (h * (self.page // 32) + t // 32) * size
            for i in (0, 1):
                for d in range(self.D):
                    b, sh = self.code_place(i, t % 32, d)
                    raw[page, at + b] = (raw[page, at + b] & ~np.uint8(15 << sh)) | np.uint8(self.c[i, page, h, t, d] << sh)
                for q in range(n):
                    for which, arr in enumerate((self.s, self.m)):
                        b = at + self.param_place(i, t % 32, q, which)
                        raw[page, b:b + 2] = np.frombuffer(arr[i, page, h, t, q].tobytes(), np.uint8)


# ---- attention ------------------------------------------------------------------------------
def attend(q, k, v, seen, scale, kind):
    """q [D], k, v [L, D] fp64, seen [L] bool -> out, lse, and their tolerances beside the
    rounding of out.

    A logit is a sum of D products of exact factors plus D/G scalings in fp32: (D + 8) steps
    of 2^-24 of sum |q| |k| at most.  Each p and each cached value is rounded to fp16 once
    (2^-11 each), exponentials and the sums of n terms are fp32."""
    D = q.shape[0]
    if not seen.any():
        return torch.zeros(D, dtype=torch.float64), -math.inf, torch.zeros(D, dtype=torch.float64), 0.0
    k, v = k[seen], v[seen]
    x = k @ q * scale
    n = x.shape[0]
    top = x.max()
    p = torch.exp(x - top)
    total = p.sum()
    w = p / total
    out = w @ v
    lse = float(top + torch.log(total))
    d = float((k.abs() @ q.abs()).max()) * scale * (D + 8) * 2.0 ** -24 + (abs(float(top)) + 40) * 2.0 ** -23
    rel = 2 * 2.0 ** -11 + 2 * d + (n + 64) * 2.0 ** -24
    return out, lse, rel * (w @ v.abs()), d + (n + 64) * 2.0 ** -24 + abs(lse) * 2.0 ** -22
