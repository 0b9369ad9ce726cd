"""Attention of video that is generated frame by frame: rotary positions, a
paged 8-bit cache of the earlier frames' keys and values, and attention over it.

One `FrameStreams` holds the cache of a batch of streams for one attention
layer. Each step takes the new tokens' projections, rotates queries and keys by
their (time, height, width) position, appends keys and values to the cache and
attends to everything cached so far:

    streams = FrameStreams(batch=1, heads=40, kv_heads=40, H=30, W=52, pages=300)
    for frame in ...:
        o, lse = streams.step(q, k, v)         # [n][heads][128] -> [heads][n][128]

The arithmetic is the library's (binding.rope_fwd, cache_write,
cache_attn_fwd); this class keeps the page table and the streams' lengths.
"""
from __future__ import annotations

from itertools import accumulate
from operator import index

import torch

from . import binding

PAGE = binding.BLOCK


class FrameStreams:
    """Cache and positions of `batch` streams of H x W frames.

    pages: pages of 128 tokens shared by the streams; max_tokens: the most
    tokens of one stream (default: all pages). A step that is refused (it needs
    more pages than are free, makes a stream longer than max_tokens, gets
    tensors or a causal_unit that do not fit) changes nothing. A step copies its lists from the host; a captured graph
    calls the binding's functions with lists of its own on the device.
    """

    def __init__(self, batch, heads, kv_heads, H, W, pages, max_tokens=None, plan=None, device=None):
        if min(batch, heads, kv_heads, H, W, pages) < 1 or heads % kv_heads:
            raise ValueError("batch, heads, kv_heads, H, W and pages must be positive, heads a multiple of kv_heads")
        if max(batch, heads) > 65535:
            raise ValueError("batch and heads must be at most 65535")
        self.batch, self.heads, self.kv_heads, self.H, self.W = batch, heads, kv_heads, H, W
        self.plan = binding.rope_plan() if plan is None else plan
        dev = torch.device("cuda" if device is None else device)
        shape = (pages, kv_heads, PAGE, binding.HEAD_DIM)
        self.k8 = torch.zeros(shape, dtype=torch.float8_e4m3fn, device=dev)
        self.v8 = torch.zeros(shape, dtype=torch.float8_e4m3fn, device=dev)
        self.k_scale = torch.ones((pages, kv_heads), dtype=torch.float32, device=dev)
        self.v_scale = torch.ones((pages, kv_heads), dtype=torch.float32, device=dev)
        self.width = pages if max_tokens is None else max(1, -(-int(max_tokens) // PAGE))
        self.table = torch.zeros((batch, self.width), dtype=torch.int32, device=dev)
        self.lengths = [0] * batch              # tokens cached by each stream
        self._owned = [[] for _ in range(batch)]  # its pages, in order
        self._free = list(range(pages - 1, -1, -1))

    @property
    def free_pages(self):
        return len(self._free)

    def _pages(self, new):
        """Pages that new[b] more tokens of each stream need, as they would be taken."""
        lengths = [n + m for n, m in zip(self.lengths, new)]
        if any(-(-n // PAGE) > self.width for n in lengths):
            raise ValueError(f"a stream would be longer than its {self.width * PAGE} tokens")
        need = [-(-n // PAGE) - len(p) for n, p in zip(lengths, self._owned)]
        if sum(need) > len(self._free):
            raise RuntimeError(f"{sum(need)} pages are needed, {len(self._free)} are free")
        at, got = len(self._free), []
        for count in need:
            got.append(self._free[at - count:at][::-1])
            at -= count
        return got

    def step(self, q, k, v, new=None, causal_unit=0):
        """Takes the new tokens' queries [n][heads][128], keys and values
        [n][kv_heads][128] (any strides), stream after stream, new[b] of each
        (default: n of the only stream); returns (o, lse), [heads][n][128] and
        [heads][n]. Tokens are frames of H x W in order; a stream goes on where
        its last step ended, inside a frame if need be. causal_unit: as in
        binding.cache_attn_fwd (H * W: a token sees its own frame and earlier
        ones; 0: all tokens of its stream, those of this step too). Made for
        generating: the outputs have no gradient."""
        n = q.shape[0]
        if new is None and self.batch == 1:
            new = [n]
        new = [] if new is None else [int(m) for m in new]
        if len(new) != self.batch or sum(new) != n or min(new) < 0:
            raise ValueError(f"new must give each of the {self.batch} streams its share of the {n} tokens")
        rest = binding.HEAD_DIM,
        if q.shape != (n, self.heads) + rest or k.shape != (n, self.kv_heads) + rest or v.shape != k.shape:
            raise ValueError(f"q must be [{n}][{self.heads}][{rest[0]}], k and v [{n}][{self.kv_heads}][{rest[0]}]")
        dev = self.k8.device
        for t, name in ((q, "q"), (k, "k"), (v, "v")):
            strides = t.stride()
            if t.dtype != torch.bfloat16 or t.device != dev or strides[2] != 1:
                raise ValueError(f"{name} must be bfloat16 on {dev} with contiguous channels")
            if n > 0 and (t.data_ptr() % 16 or strides[0] % 8 or strides[1] % 8):
                raise ValueError(f"{name} must begin on 16 bytes, and so must its rows")
        causal_unit = index(causal_unit)
        if not 0 <= causal_unit < 1 << 31:
            raise ValueError("causal_unit must be a number of tokens, or 0")
        rows = max(new) * (self.heads // self.kv_heads)  # the attention's limits
        if rows >= 1 << 30 or max(1, -(-rows // 256)) * self.batch * self.kv_heads >= 1 << 30:
            raise ValueError("more tokens than one step takes")
        got = self._pages(new)
        hw = self.H * self.W
        lengths = [a + m for a, m in zip(self.lengths, new)]
        lists = torch.tensor([0, *accumulate(new), *lengths], dtype=torch.int32)
        if self.batch == 1 and self.lengths[0] % hw == 0:
            where = dict(grid=(self.H, self.W), start=(self.lengths[0] // hw, 0, 0))
            start, length = lists.to(dev).split((self.batch + 1, self.batch))
        else:
            t = torch.cat([torch.arange(a, a + m) for a, m in zip(self.lengths, new)])
            pos = torch.stack([t // hw, t % hw // self.W, t % self.W], 1).to(torch.int32)
            lists = torch.cat([pos.view(-1), lists]).to(dev)  # one copy
            pos, start, length = lists.split((3 * n, self.batch + 1, self.batch))
            where = dict(pos=pos.view(n, 3))
        q, k = binding.rope_fwd(q.detach(), k.detach(), self.plan, **where)
        for b, pages in enumerate(got):
            if pages:
                at = len(self._owned[b])
                self.table[b, at:at + len(pages)] = torch.tensor(pages, dtype=torch.int32, device=dev)
        # nothing that the arguments or the host's state decide is refused from here on
        binding.cache_write(k.transpose(0, 1), v, self.k8, self.v8, self.k_scale, self.v_scale, start, length,
                            self.table, max_new=max(new))
        out = binding.cache_attn_fwd(q, self.k8, self.v8, self.k_scale, self.v_scale, start, length, self.table,
                                     max_new=max(new), max_kv=max(lengths), causal_unit=causal_unit)
        del self._free[len(self._free) - sum(map(len, got)):]
        for pages, owned in zip(got, self._owned):
            owned += pages
        self.lengths = lengths
        return out

    def drop(self, b):
        """Ends stream b: its pages are free again and it starts anew."""
        self._free += reversed(self._owned[b])
        self._owned[b] = []
        self.lengths[b] = 0
