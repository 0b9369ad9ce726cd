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

import torch

from . import binding

PAGE = binding.BLOCK


class FrameStreams:
    """Cache and positions of `batch` streams of H x W frames.

    pages: pages of 128 tokens shared by the streams; max_tokens: the most
    tokens of one stream (default: all pages). A step that needs more pages
    than are free, or makes a stream longer than max_tokens, is refused before
    anything is changed. A step copies its lists from the host; a captured graph
    calls the binding's functions with lists of its own on the device.
    """

    def __init__(self, batch, heads, kv_heads, H, W, pages, max_tokens=None, plan=None, device=None):
        if min(batch, heads, kv_heads, H, W, pages) < 1 or heads % kv_heads:
            raise ValueError("batch, heads, kv_heads, H, W and pages must be positive, heads a multiple of kv_heads")
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

    def _extend(self, new):
        """Pages for new[b] more tokens of each stream."""
        need = [-(-(n + m) // PAGE) - len(p) for n, m, p in zip(self.lengths, new, self._owned)]
        if any(-(-(n + m) // PAGE) > self.width for n, m in zip(self.lengths, new)):
            raise ValueError(f"a stream would be longer than its {self.width * PAGE} tokens")
        if sum(need) > len(self._free):
            raise RuntimeError(f"{sum(need)} pages are needed, {len(self._free)} are free")
        for b, count in enumerate(need):
            if count > 0:
                got = [self._free.pop() for _ in range(count)]
                at = len(self._owned[b])
                self._owned[b] += got
                self.table[b, at:at + count] = torch.tensor(got, dtype=torch.int32, device=self.table.device)

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
        for t, name in ((q, "q"), (k, "k"), (v, "v")):
            if t.dtype != torch.bfloat16 or t.device != self.k8.device or t.stride(2) != 1:
                raise ValueError(f"{name} must be bfloat16 on {self.k8.device} with contiguous channels")
        self._extend(new)
        dev = self.k8.device
        hw = self.H * self.W
        if self.batch == 1 and self.lengths[0] % hw == 0:
            where = dict(grid=(self.H, self.W), start=(self.lengths[0] // hw, 0, 0))
        else:
            t = torch.cat([torch.arange(a, a + m) for a, m in zip(self.lengths, new)])
            where = dict(pos=torch.stack([t // hw, t % hw // self.W, t % self.W], 1).to(torch.int32).to(dev))
        with torch.no_grad():
            q, k = binding.rope_fwd(q, k, self.plan, **where)
        lengths = [a + m for a, m in zip(self.lengths, new)]
        start = torch.tensor([0] + new, dtype=torch.int32).cumsum(0, dtype=torch.int32).to(dev)
        length = torch.tensor(lengths, dtype=torch.int32).to(dev)
        binding.cache_write(k.transpose(0, 1), v, self.k8, self.v8, self.k_scale, self.v_scale, start, length,
                            self.table, max_new=max(new))
        out = binding.cache_attn_fwd(q, self.k8, self.v8, self.k_scale, self.v_scale, start, length, self.table,
                                     max_new=max(new), max_kv=max(lengths), causal_unit=causal_unit)
        self.lengths = lengths
        return out

    def drop(self, b):
        """Ends stream b: its pages are free again and it starts anew."""
        self._free += reversed(self._owned[b])
        self._owned[b] = []
        self.lengths[b] = 0
