"""Plain definitions, in 64 bits and whole numbers on the CPU, of the operators around drafted trees:
masks and depths, attention, pages forked and tokens compacted, rotary positions.  Written from the
formulas in include/w4a16.h; shares no code with the library."""
import math

import numpy as np
import torch

import decoder_ref as ref


# ---- trees ----------------------------------------------------------------------------------
def branches(parents):
    """The nodes that each node follows, itself first."""
    out = []
    for i, p in enumerate(parents):
        out.append([i] + (out[p] if 0 <= p < i else []))
    return out


def mask_rows(lines, words, window=0):
    m = np.zeros((len(lines), words), np.uint32)
    for i, line in enumerate(lines):
        for j in line[:window] if window else line:
            m[i, j // 32] |= np.uint32(1 << (j % 32))
    return m


def trees(r, kind, n):
    """Parents of n nodes."""
    if kind == "chain":
        return [i - 1 for i in range(n)]
    if kind == "star":
        return [-1] + [0] * (n - 1) if n else []
    if kind == "forest":
        return [-1 if r.random() < 0.3 else r.randrange(i) if i else -5 for i in range(n)]
    return [r.randrange(max(0, i - 6), i) if i else -1 for i in range(n)]


# ---- the 4-bit pages ---------------------------------------------------------------------------
class Bytes:
    """Where a token's bytes lie in a block of 32 tokens (as tests/decoder_ref.py has it)."""

    def __init__(self, heads, D, G, page):
        c = ref.Cache(1, heads, D, G, page)
        self.heads, self.D, self.G, self.page, self.size = heads, D, G, page, c.block_bytes()
        self.code = np.array([[[c.code_place(i, t, d) for d in range(D)] for t in range(32)] for i in (0, 1)])
        self.par = np.array([[[c.param_place(i, t, q, w) for q in range(D // G) for w in (0, 1)] for t in range(32)] for i in (0, 1)])

    def blocks(self, raw):
        """raw [pages, bytes] -> view [pages, heads, blocks, size]."""
        return raw.reshape(raw.shape[0], self.heads, self.page // 32, self.size)

    def take(self, blocks, page, at):
        """Codes [heads, 2, D] and parameters [heads, 2, 2 D/G] of the token at a place of a page."""
        x = blocks[page, :, at // 32]
        t = at % 32
        codes = np.stack([(x[:, self.code[i, t, :, 0]] >> self.code[i, t, :, 1].astype(np.uint8)) & 15 for i in (0, 1)], 1)
        par = np.stack([np.ascontiguousarray(x).view(np.uint16)[:, self.par[i, t] // 2] for i in (0, 1)], 1)
        return codes, par

    def put(self, blocks, page, at, codes, par):
        x = blocks[page, :, at // 32]
        t = at % 32
        for i in (0, 1):
            b, sh = self.code[i, t, :, 0], self.code[i, t, :, 1].astype(np.uint8)
            for d in range(self.D):  # two channels or tokens share a byte
                x[:, b[d]] = (x[:, b[d]] & ~np.uint8(15 << sh[d])) | (codes[:, i, d] << sh[d]).astype(np.uint8)
            for j, at2 in enumerate(self.par[i, t]):
                x[:, at2] = par[:, i, j] & 255
                x[:, at2 + 1] = par[:, i, j] >> 8

    def values(self, raw):
        """[2, pages, heads, page, D] in fp64."""
        x = self.blocks(raw)
        out = np.empty((2,) + x.shape[:3] + (32, self.D))
        h = np.ascontiguousarray(x).view(np.float16)
        with np.errstate(invalid="ignore", over="ignore"):
            for i in (0, 1):
                for t in range(32):
                    c = (x[..., self.code[i, t, :, 0]] >> self.code[i, t, :, 1].astype(np.uint8)) & 15
                    p = h[..., self.par[i, t] // 2].astype(np.float64)
                    out[i, ..., t, :] = np.repeat(p[..., 1::2], self.G, -1) + np.repeat(p[..., 0::2], self.G, -1) * c
        return out.reshape(2, x.shape[0], self.heads, self.page, self.D)


# ---- attention ----------------------------------------------------------------------------------
def attend(q, k, v, seen, scale):
    """q [R, D], k, v [L, D] fp64, seen [R, L] -> out, lse and their tolerances beside the rounding of
    out: the arithmetic that tests/decoder_ref.py's attend derives, for many rows at once."""
    D, L = q.shape[1], k.shape[0]
    n = seen.sum(1)
    some = seen.any(0)
    k, v = torch.where(some[:, None], k, 0.0), torch.where(some[:, None], v, 0.0)
    x = (q @ k.t() * scale).masked_fill(~seen, -math.inf)
    top = x.amax(1) if L else torch.full((len(q),), -math.inf, dtype=torch.float64)
    none = n == 0
    safe = torch.where(none, 0.0, top)
    p = torch.exp(x - safe[:, None])
    total = p.sum(1)
    w = p / torch.where(none, 1.0, total)[:, None]
    out = w @ v
    lse = torch.where(none, -math.inf, safe + torch.log(torch.where(none, 1.0, total)))
    reach = (q.abs() @ k.abs().t()).masked_fill(~seen, 0.0).amax(1) if L else torch.zeros(len(q))
    d = reach * scale * (D + 8) * 2.0 ** -24 + (safe.abs() + 40) * 2.0 ** -23
    rel = 2 * 2.0 ** -11 + 2 * d + (n + 64) * 2.0 ** -24
    ltol = d + (n + 64) * 2.0 ** -24 + torch.where(none, 0.0, lse).abs() * 2.0 ** -22
    return out, lse, rel[:, None] * (w @ v.abs()), ltol


# ---- pages --------------------------------------------------------------------------------------
def fork(table, lens, parent, keep, room, pinned, pages, page):
    """New table, lens, missing, and the copies: (from, to, tokens)."""
    W = len(table[0])
    ok = lambda p: 0 <= p < pages  # noqa: E731
    rows = []
    for r, p in enumerate(parent):
        has = max(0, lens[p]) if 0 <= p < len(table) else 0
        k = min(max(0, has if keep is None else min(keep[r], has)), W * page)
        m = min(max(k, room[r] if room is not None else 0), W * page)
        rows.append((p, k, m))
    held = {i for i in range(pages) if pinned is not None and pinned[i]}
    for p, k, _ in rows:
        held.update(x for x in (table[p][:k // page] if k else []) if ok(x))
    mine = {}
    for r, (p, k, _) in enumerate(rows):
        if k % page and ok(table[p][k // page]) and table[p][k // page] not in held:
            mine.setdefault(table[p][k // page], r)
    free = iter(sorted(set(range(pages)) - held - set(mine)))
    out, copies, missing = [], [], 0
    for r, (p, k, m) in enumerate(rows):
        row = [x if ok(x) else -1 for x in table[p][:k // page]] if k else []
        if k % page:
            old = table[p][k // page]
            if not ok(old):
                row.append(-1)
            elif mine.get(old) == r:
                row.append(old)
            else:
                new = next(free, -1)
                missing += new < 0
                if new >= 0:
                    copies.append((old, new, k % page))
                row.append(new)
        while len(row) * page < m:
            new = next(free, -1)
            missing += new < 0
            row.append(new)
        out.append(row + [-1] * (W - len(row)))
    return out, [k for _, k, _ in rows], missing, copies


# ---- rotary ---------------------------------------------------------------------------------------
def rotary(x, heads, pos, axis, freq, neighbours):
    """x [tokens, heads * head] -> y in fp64 and the error it may have beside its rounding: angles and
    their cosines in fp32 are off by 2^-20 at most, and by 2^-51 of the angle formed in 64 bits."""
    T, half = x.shape[0], len(freq)
    a64 = pos[axis].double() * freq.double()[:, None]
    c, s = torch.cos(a64).t()[:, None], torch.sin(a64).t()[:, None]
    y = x.double().view(T, heads, -1).clone()
    i = torch.arange(half)
    a, b = (2 * i, 2 * i + 1) if neighbours else (i, i + half)
    p, q = y[..., a].clone(), y[..., b].clone()
    y[..., a], y[..., b] = p * c - q * s, q * c + p * s
    tol = torch.zeros_like(y)
    tol[..., a] = tol[..., b] = (p.abs() + q.abs()) * (2.0 ** -20 + a64.abs().t()[:, None] * 2.0 ** -51)
    return y.view(T, -1), tol.view(T, -1)
