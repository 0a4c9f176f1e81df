"""The operators of one decoder step over the 4-bit products: a cache of keys and values
held in 4 bits, trees of drafted tokens over it and the pages of all layers, rotary
positions, and the attention half of a decoder layer that runs norm, products, adapters,
cache and attention together.  Like the linear layers (layer.py) these classes do
no arithmetic of their own: they check shapes and forward to the library.  They are for
inference: no gradient passes through any of them."""
from __future__ import annotations

import torch

from . import (DT_BF16, DT_F16, ROTARY_HALVES, ROTARY_NEIGHBOURS, w4a8_rmsnorm, w4a16_kv4_append,
               w4a16_kv4_attention, w4a16_kv4_compact, w4a16_kv4_fork, w4a16_kv4_gather,
               w4a16_kv4_page_bytes, w4a16_kv4_tree, w4a16_kv4_tree_attention, w4a16_lora,
               w4a16_rotary)
from .layer import W4A16Linear

_TYPES = {torch.float16: DT_F16, torch.bfloat16: DT_BF16}


def _rows16(name: str, x: torch.Tensor, width: int) -> int:
    """The distance between the rows of a 16-bit [rows, width] tensor with unit stride inside."""
    if x.dtype not in _TYPES:
        raise TypeError(f"{name}: expected float16 or bfloat16, got {x.dtype}")
    if x.dim() != 2 or x.shape[1] != width or (width > 1 and x.stride(1) != 1):
        raise ValueError(f"{name}: expected rows of {width} values side by side, got {tuple(x.shape)}")
    return x.stride(0) if x.shape[0] > 1 else width


def _ints(name: str, x: torch.Tensor, *shape: int, dtype: torch.dtype = torch.int32) -> None:
    if x.dtype != dtype or not x.is_contiguous() or tuple(x.shape) != shape:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape}")


def _one_gpu(*tensors: torch.Tensor | None) -> None:
    """Refuses tensors that are not all on the current GPU: the kernels get bare addresses."""
    here = tensors[0].device
    if here.type != "cuda" or here.index != torch.cuda.current_device():
        raise ValueError(f"the tensors must be on the current GPU, not on device {here}")
    for x in tensors:
        if x is not None and x.device != here:
            raise ValueError(f"the tensors of a call must be on one device, not on {here} and {x.device}")


class Batch:
    """The sequences of one step: `rows` int32 [batch + 1] (sequence b's new tokens are rows
    rows[b] .. rows[b + 1] - 1 of q, k and v), `lens` int32 [batch] (lengths with the new
    tokens), `table` int32 [batch, width] (pages, -1: none), all on the device; `max_new`
    and `max_len` bound the new tokens and the length of a sequence on the host."""

    def __init__(self, rows: torch.Tensor, lens: torch.Tensor, table: torch.Tensor, max_new: int,
                 max_len: int):
        for name, x in (("rows", rows), ("lens", lens), ("table", table)):
            if x.dtype != torch.int32 or not x.is_contiguous():
                raise TypeError(f"{name} must be a contiguous int32 tensor")
        if lens.dim() != 1 or table.dim() != 2 or tuple(rows.shape) != (lens.shape[0] + 1,) or table.shape[0] != lens.shape[0]:
            raise ValueError("rows must be [batch + 1], lens [batch] and table [batch, width]")
        self.rows, self.lens, self.table = rows, lens, table
        self.size, self.max_new, self.max_len = lens.shape[0], max_new, max_len


class Tree:
    """The drafted tokens of a step as trees, one for each sequence of `batch`, whose new tokens
    are the nodes: `parent` int32 [tokens] on the device, the node of the same sequence that each
    follows (below 0: the last token held before).  From it `mask` (bits of the nodes that each
    sees), `depth` and `pos` (its position in the sequence, for Rotary).  `window`: how many tokens
    back a token sees, itself included (0: all)."""

    def __init__(self, parent: torch.Tensor, batch: Batch, window: int = 0):
        if parent.dim() != 1:
            raise ValueError("parent must be [tokens]")
        n = parent.shape[0]
        _ints("parent", parent, n)
        most = max(1, min(batch.max_new, n))
        self.words, self.window = (most + 31) // 32, window
        # rows of no sequence, which the kernel does not write, see nothing
        self.mask = torch.zeros((n, self.words), dtype=torch.int32, device=parent.device)
        self.depth, self.pos = torch.zeros((2, n), dtype=torch.int32, device=parent.device)
        if n > 0:
            _one_gpu(parent, batch.rows, batch.lens)
            w4a16_kv4_tree(parent, batch.rows, batch.lens, self.mask, self.depth, self.pos, batch.size, n, most,
                           self.words, window)


class Rotary(torch.nn.Module):
    """Rotary positions: pair i of a head's first 2 * len(freq) channels, (i, i + len(freq)) or with
    `neighbours` (2 i, 2 i + 1), is turned by pos * freq[i], on the axis axis[i] where positions
    have several (time, height, width); freq fp32, axis int32."""

    def __init__(self, freq: torch.Tensor, head: int, axis: torch.Tensor | None = None, neighbours: bool = False):
        super().__init__()
        if freq.dim() != 1 or freq.dtype != torch.float32:
            raise TypeError("freq must be float32 [pairs]")
        n = freq.shape[0]
        if n < 8 or n % 8 or 2 * n > head or head % 8 or head > 512:
            raise ValueError(f"unsupported: {n} pairs (a multiple of 8) of {head} channels (a multiple of 8, at most 512)")
        if axis is not None:
            _ints("axis", axis, n)
        self.head, self.neighbours = head, neighbours
        self.register_buffer("freq", freq.contiguous())
        self.register_buffer("axis", axis)

    def _apply(self, fn, recurse=True):
        # half(), bfloat16() and their like are not about the frequencies: they stay fp32, bit for bit
        freq = self.freq
        super()._apply(fn, recurse)
        if self.freq.dtype != freq.dtype:
            self.freq = freq.to(self.freq.device)
        return self

    def forward(self, q: torch.Tensor, k: torch.Tensor | None, pos: torch.Tensor) -> None:
        """Turns q [tokens, q_heads * head] and k (may be None) in place; pos int32 [tokens] or
        [axes, tokens]."""
        axes = 1 if pos.dim() == 1 else pos.shape[0]
        _ints("pos", pos, *((q.shape[0],) if pos.dim() == 1 else (axes, q.shape[0])))
        if axes < 1 or (axes > 1 and self.axis is None):
            raise ValueError("positions with several axes need an axis for each frequency")
        if self.freq.dtype != torch.float32 or not self.freq.is_contiguous():  # buffers can have changed
            raise TypeError("freq must be contiguous float32")
        ld, heads = [], []
        for name, x in (("q", q), ("k", k)):
            if x is None:
                ld.append(0)
                heads.append(0)
                continue
            if x.dim() != 2 or x.shape[1] % self.head or x.shape[1] == 0 or x.shape[0] != q.shape[0] or x.dtype != q.dtype:
                raise ValueError(f"{name} must be [tokens, heads * {self.head}], as many rows and of the same type as q")
            ld.append(_rows16(name, x, x.shape[1]))
            heads.append(x.shape[1] // self.head)
            if x.requires_grad and torch.is_grad_enabled():
                raise ValueError(f"{name} requires a gradient, which would not see that it is turned in place")
        if q.shape[0] > 0:
            _one_gpu(self.freq, self.axis, pos, q, k)
            w4a16_rotary(q, k, pos, self.axis, self.freq, q, k, q.shape[0], *heads, self.head, 2 * self.freq.shape[0], axes,
                         q.shape[0], *ld, *ld, ROTARY_NEIGHBOURS if self.neighbours else ROTARY_HALVES, _TYPES[q.dtype])

    def at(self, pos: torch.Tensor):
        """The `rotate` of AttentionBlock for tokens at these positions."""
        return lambda q, k: self(q, k, pos)


class Kv4Cache(torch.nn.Module):
    """Pages of keys and values in 4 bits, `page` tokens of every kv head each; codes with an
    fp16 scale and minimum per token, kv head and `group` channels (w4a16_kv4_append).  `data`:
    the pages, where they are a layer of a Kv4Pool."""

    def __init__(self, pages: int, kv_heads: int, head: int, group: int = 64, page: int = 64, device="cuda",
                 data: torch.Tensor | None = None):
        super().__init__()
        size = w4a16_kv4_page_bytes(kv_heads, head, group, page)
        if size == 0 or pages < 1:
            raise ValueError(f"unsupported layout: pages={pages}, kv_heads={kv_heads}, head={head} (64 or 128), "
                             f"group={group} (32, 64 or 128, at most head), page={page} (a multiple of 32)")
        self.pages, self.kv_heads, self.head, self.group, self.page = pages, kv_heads, head, group, page
        # contents of a moment, sized by the machine: moved with the model, but not saved with it
        self.of_pool = data is not None
        if data is not None:
            _ints("data", data, pages, size, dtype=torch.uint8)
        else:
            data = torch.empty((pages, size), dtype=torch.uint8, device=device)
        self.register_buffer("data", data, persistent=False)

    def _apply(self, fn, recurse=True):
        return self if self.of_pool else super()._apply(fn, recurse)  # the pool moves its layers' pages

    def _load_from_state_dict(self, state_dict, prefix, *args):
        state_dict.pop(prefix + "data", None)  # checkpoints that hold the pages of their moment
        super()._load_from_state_dict(state_dict, prefix, *args)

    def _layout(self, batch: Batch):
        return self.kv_heads, self.head, self.group, self.page, self.pages, batch.table.shape[1]

    def _kv(self, k, v):
        width = self.kv_heads * self.head
        ldk, ldv = _rows16("k", k, width), _rows16("v", v, width)
        if k.shape[0] != v.shape[0] or k.dtype != v.dtype:
            raise ValueError("k and v must have the same rows and type")
        return ldk, ldv

    def append(self, k: torch.Tensor, v: torch.Tensor, batch: Batch) -> None:
        """Quantizes the new tokens' k and v [tokens, kv_heads * head] into their pages."""
        ldk, ldv = self._kv(k, v)
        if k.shape[0] > 0:
            _one_gpu(self.data, k, v, batch.rows, batch.lens, batch.table)
            w4a16_kv4_append(k, v, batch.rows, batch.lens, batch.table, self.data, batch.size, k.shape[0],
                             min(batch.max_new, k.shape[0]), ldk, ldv, *self._layout(batch), _TYPES[k.dtype])

    def gather(self, k: torch.Tensor, v: torch.Tensor, batch: Batch) -> None:
        """Writes the cached values of the same tokens to the rows of k and v."""
        ldk, ldv = self._kv(k, v)
        if k.shape[0] > 0:
            _one_gpu(self.data, k, v, batch.rows, batch.lens, batch.table)
            w4a16_kv4_gather(self.data, batch.rows, batch.lens, batch.table, k, v, batch.size, k.shape[0],
                             min(batch.max_new, k.shape[0]), ldk, ldv, *self._layout(batch), _TYPES[k.dtype])

    def attend(self, q: torch.Tensor, batch: Batch, q_heads: int, window: int = 0, scale: float | None = None,
               lse: torch.Tensor | None = None) -> torch.Tensor:
        """Attention of the new tokens q [tokens, q_heads * head] over the cached ones.  Rows of
        no sequence (padding, new tokens past batch.max_new) are 0; in lse they keep what they held.
        Single tokens with long contexts are faster in a batch of their own than beside a prompt."""
        ldq = _rows16("q", q, q_heads * self.head)
        if lse is not None and (lse.dtype != torch.float32 or tuple(lse.shape) != (q.shape[0], q_heads) or not lse.is_contiguous()):
            raise ValueError(f"lse must be a contiguous float32 tensor of shape {(q.shape[0], q_heads)}")
        # which rows have a sequence is known on the device only, and the kernel writes no others
        out = torch.zeros((q.shape[0], q_heads * self.head), dtype=q.dtype, device=q.device)
        if q.shape[0] > 0:
            _one_gpu(self.data, q, batch.rows, batch.lens, batch.table, lse)
            w4a16_kv4_attention(q, batch.rows, batch.lens, batch.table, self.data, out, lse, batch.size, q.shape[0],
                                min(batch.max_new, q.shape[0]), batch.max_len, ldq, q_heads * self.head, q_heads,
                                *self._layout(batch), window, self.head ** -0.5 if scale is None else scale,
                                _TYPES[q.dtype])
        return out

    def attend_tree(self, q: torch.Tensor, batch: Batch, tree: Tree, q_heads: int, scale: float | None = None,
                    lse: torch.Tensor | None = None) -> torch.Tensor:
        """Attention of the nodes of drafted trees, q [tokens, q_heads * head], over the tokens cached
        before them and each node's own branch (append them first).  Rows of no sequence are 0."""
        ldq = _rows16("q", q, q_heads * self.head)
        if tree.mask.shape[0] != q.shape[0]:
            raise ValueError("the tree must have a node for each row of q")
        if 32 * tree.words < min(batch.max_new, q.shape[0]):
            raise ValueError("the tree must be of this batch")
        if lse is not None and (lse.dtype != torch.float32 or tuple(lse.shape) != (q.shape[0], q_heads) or not lse.is_contiguous()):
            raise ValueError(f"lse must be a contiguous float32 tensor of shape {(q.shape[0], q_heads)}")
        out = torch.zeros((q.shape[0], q_heads * self.head), dtype=q.dtype, device=q.device)
        if q.shape[0] > 0:
            _one_gpu(self.data, q, batch.rows, batch.lens, batch.table, tree.mask, tree.depth, lse)
            w4a16_kv4_tree_attention(q, batch.rows, batch.lens, batch.table, self.data, tree.mask, tree.depth, out, lse,
                                     batch.size, q.shape[0], min(batch.max_new, q.shape[0]), batch.max_len, tree.words, ldq,
                                     q_heads * self.head, q_heads, *self._layout(batch), tree.window,
                                     self.head ** -0.5 if scale is None else scale, _TYPES[q.dtype])
        return out


class Kv4Pool(torch.nn.Module):
    """The caches of a model's layers, which share one table of pages: pool[i] is the Kv4Cache of
    layer i.  What is done with pages as such is done for all layers at once."""

    def __init__(self, layers: int, pages: int, kv_heads: int, head: int, group: int = 64, page: int = 64, device="cuda"):
        super().__init__()
        size = w4a16_kv4_page_bytes(kv_heads, head, group, page)
        if size == 0 or pages < 1 or layers < 1:
            raise ValueError(f"unsupported layout: layers={layers}, pages={pages}, kv_heads={kv_heads}, head={head}, group={group}, page={page}")
        self.pages, self.page = pages, page
        self.layout = kv_heads, head, group, page, pages
        self.register_buffer("data", torch.empty((layers, pages, size), dtype=torch.uint8, device=device), persistent=False)
        self.caches = torch.nn.ModuleList(Kv4Cache(pages, kv_heads, head, group, page, data=self.data[i]) for i in range(layers))

    def _apply(self, fn, recurse=True):
        super()._apply(fn, recurse)
        for i, cache in enumerate(self.caches):
            cache.data = self.data[i]
        return self

    def __getitem__(self, layer: int) -> Kv4Cache:
        return self.caches[layer]

    def __len__(self) -> int:
        return len(self.caches)

    def compact(self, path: torch.Tensor, count: torch.Tensor, batch: Batch) -> torch.Tensor:
        """Keeps of each sequence's drafted tree the count[b] nodes path[b] (int32 [batch, most],
        ascending along the branch), behind the tokens held before; returns the new lengths."""
        if path.dim() != 2 or path.shape[1] < 1:
            raise ValueError("path must be [batch, most]")
        _ints("path", path, batch.size, path.shape[1])
        _ints("count", count, batch.size)
        lens = torch.empty_like(batch.lens)
        _one_gpu(self.data, path, count, batch.rows, batch.lens, batch.table)
        # rows of sequences say how many nodes there are, whatever the number of tokens behind them
        w4a16_kv4_compact(self.data, path, count, batch.rows, batch.lens, batch.table, lens, batch.size, (1 << 31) - 1,
                          batch.max_new, path.shape[1], len(self), self.data.stride(0), *self.layout, batch.table.shape[1])
        return lens

    def fork(self, table: torch.Tensor, lens: torch.Tensor, parent: torch.Tensor, keep: torch.Tensor | None = None,
             room: torch.Tensor | None = None, pinned: torch.Tensor | None = None):
        """Who has which pages in the next step (w4a16_kv4_fork): row r of the new table goes on from
        row parent[r] (below 0: from nothing), keeps keep[r] of its tokens (None: all) and has pages
        for room[r] tokens; pinned uint8 [pages] are not given out.  Returns table, lens and how many
        pages were missing (int32 [1]).  Where that is above 0 the old table still holds for what these
        rows keep: call again with fewer of them, or with less kept or less room.  Pages that none of
        them keeps and that are not pinned may have been written already."""
        if table.dim() != 2 or parent.dim() != 1 or parent.shape[0] < 1:
            raise ValueError("table must be [batch, width] and parent [rows]")
        n = parent.shape[0]
        _ints("table", table, *table.shape)
        _ints("lens", lens, table.shape[0])
        _ints("parent", parent, n)
        for name, x in (("keep", keep), ("room", room)):
            if x is not None:
                _ints(name, x, n)
        if pinned is not None:
            _ints("pinned", pinned, self.pages, dtype=torch.uint8)
        _one_gpu(self.data, table, lens, parent, keep, room, pinned)
        new = torch.empty((n, table.shape[1]), dtype=torch.int32, device=table.device)
        held = torch.empty(n, dtype=torch.int32, device=table.device)
        missing = torch.empty(1, dtype=torch.int32, device=table.device)
        w4a16_kv4_fork(self.data, table, lens, parent, keep, room, pinned, new, held, missing, table.shape[0], n, len(self),
                       self.data.stride(0), *self.layout, table.shape[1])
        return new, held, missing


class Adapters(torch.nn.Module):
    """Low-rank adapters beside one projection: y[m] += scale[a] * (x[m] A[a]^T) B[a]^T, in
    place, a = ids[m] (below 0: none)."""

    def __init__(self, A: torch.Tensor, B: torch.Tensor, scale: torch.Tensor):
        super().__init__()
        if A.dim() != 3 or B.dim() != 3 or A.shape[0] != B.shape[0] or A.shape[1] != B.shape[2] or tuple(scale.shape) != (A.shape[0],):
            raise ValueError("A must be [adapters, rank, in], B [adapters, out, rank] and scale [adapters]")
        if A.dtype != B.dtype or A.dtype not in _TYPES or scale.dtype != torch.float32:
            raise TypeError("A and B must both be float16 or bfloat16, scale float32")
        for name, x in (("A", A), ("B", B), ("scale", scale)):
            self.register_buffer(name, x.contiguous())

    def _apply(self, fn, recurse=True):
        # half(), bfloat16() and their like are about A and B: scale stays fp32, bit for bit
        scale = self.scale
        super()._apply(fn, recurse)
        if self.scale.dtype != scale.dtype:
            self.scale = scale.to(self.scale.device)
        return self

    def forward(self, x: torch.Tensor, y: torch.Tensor, ids: torch.Tensor) -> torch.Tensor:
        # buffers can have changed since they were checked
        if self.A.dtype not in _TYPES or self.B.dtype != self.A.dtype or self.scale.dtype != torch.float32:
            raise TypeError(f"A and B must both be float16 or bfloat16 and scale float32, not {self.A.dtype}, {self.B.dtype} and {self.scale.dtype}")
        if not (self.A.is_contiguous() and self.B.is_contiguous() and self.scale.is_contiguous()):
            raise ValueError("A, B and scale must be contiguous")
        adapters, rank, K = self.A.shape
        N = self.B.shape[1]
        ldx, ldy = _rows16("x", x, K), _rows16("y", y, N)
        if x.dtype != self.A.dtype or y.dtype != x.dtype or x.shape[0] != y.shape[0]:
            raise ValueError("x and y must have the same rows and the adapters' type")
        if ids.dtype != torch.int32 or tuple(ids.shape) != (x.shape[0],) or not ids.is_contiguous():
            raise ValueError(f"ids must be a contiguous int32 tensor of {x.shape[0]} values")
        if y.requires_grad and torch.is_grad_enabled():
            raise ValueError("y requires a gradient, which would not see what is added in place")
        if x.shape[0] > 0:
            _one_gpu(self.A, self.B, self.scale, x, y, ids)
            w4a16_lora(x, self.A, self.B, ids, self.scale, y, y, x.shape[0], N, K, rank, adapters, ldx, ldy,
                       _TYPES[x.dtype])
        return y


class AttentionBlock(torch.nn.Module):
    """The attention half of a decoder layer in fp16:

        h = x + residual;  n = norm(h), 8-bit rows;  q, k, v = n Wqkv (+ adapters)
        cache <- k, v;  o = attention(q, cache);  y = o Wo (+ adapters)

    forward returns (y, h).  `rotate(q, k)`, if given, turns q and k in place before they are
    used (positions are the caller's: Rotary.at).  With `tree` the new tokens are the nodes of
    drafted trees, and attend by it."""

    def __init__(self, gamma: torch.Tensor, qkv: W4A16Linear, out: W4A16Linear, cache: Kv4Cache, q_heads: int,
                 eps: float = 1e-5, qkv_adapters: Adapters | None = None, out_adapters: Adapters | None = None):
        super().__init__()
        width = (q_heads + 2 * cache.kv_heads) * cache.head
        if q_heads < 1 or q_heads % cache.kv_heads:
            raise ValueError("q_heads must be a multiple of the cache's kv_heads")
        if qkv.out_features != width or out.in_features != q_heads * cache.head or tuple(gamma.shape) != (qkv.in_features,):
            raise ValueError(f"qkv must have {width} outputs, out {q_heads * cache.head} inputs and gamma one value per input of qkv")
        if gamma.dtype != torch.float16:
            raise TypeError("gamma must be float16")
        self.register_buffer("gamma", gamma.contiguous())
        self.qkv, self.out, self.cache = qkv, out, cache
        self.qkv_adapters, self.out_adapters = qkv_adapters, out_adapters
        self.q_heads, self.eps = q_heads, eps

    def forward(self, x: torch.Tensor, residual: torch.Tensor | None, batch: Batch, ids: torch.Tensor | None = None,
                window: int = 0, rotate=None, tree: Tree | None = None):
        if tree is not None and window != tree.window:
            raise ValueError("window must be that of the tree")
        K = self.qkv.in_features
        if x.dtype != torch.float16 or x.dim() != 2 or x.shape[1] != K:
            raise ValueError(f"x must be float16 [tokens, {K}]")
        if residual is not None and (residual.dtype != x.dtype or residual.shape != x.shape):
            raise ValueError("residual must be like x")
        if self.gamma.dtype != x.dtype or not self.gamma.is_contiguous():  # a cast of the model reaches it
            raise TypeError(f"gamma must be contiguous float16, not {self.gamma.dtype}")
        x = x.contiguous()
        M = x.shape[0]
        h = torch.empty_like(x)
        y8 = torch.empty((M, K), dtype=torch.float8_e4m3fn, device=x.device)
        scale = torch.empty(M, dtype=torch.float32, device=x.device)
        adapt = ids is not None and self.qkv_adapters is not None
        n = torch.empty_like(x) if adapt else None
        if M == 0:
            return torch.empty((0, self.out.out_features), dtype=x.dtype, device=x.device), h
        _one_gpu(x, residual, self.gamma, self.qkv.wp, self.out.wp)
        w4a8_rmsnorm(x, None if residual is None else residual.contiguous(), self.gamma, h, y8, scale, n, M, K, self.eps, DT_F16)
        qkv = self.qkv(y8, scale)
        if adapt:
            self.qkv_adapters(n, qkv, ids)
        kv = self.cache.kv_heads * self.cache.head
        q, k, v = qkv.split([self.q_heads * self.cache.head, kv, kv], 1)
        if rotate is not None:
            rotate(q, k)
        self.cache.append(k, v, batch)
        if tree is None:
            o = self.cache.attend(q, batch, self.q_heads, window)
        else:
            o = self.cache.attend_tree(q, batch, tree, self.q_heads)
        y = self.out(o)
        if ids is not None and self.out_adapters is not None:
            self.out_adapters(o, y, ids)
        return y, h
