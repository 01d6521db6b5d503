"""A paged cache on the GPU and what its calls should make of it, for the tests."""
from __future__ import annotations

import numpy as np
import torch

from layer_helpers import LEAST, TORCH

E4M3 = torch.float8_e4m3fn


class Cache:
    """Pools filled with codes or values from `seed`, a table that deals out shuffled pages
    (-1 where a sequence has none), scales.  gap: elements between pages.  One buffer
    holds the pages of k and v in turn when `both` is set."""

    def __init__(self, lens, heads, D, page, dtype, cache, seed=0, gap=0, both=False, spare=2,
                 width=None, extra_columns=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens_host, self.heads, self.D, self.page = list(lens), heads, D, page
        self.dtype, self.cache, self.B = dtype, cache, len(lens)
        need = [-(-max(n, 0) // page) for n in lens]
        self.width = width or max([1] + need)
        self.pages = sum(need) + spare
        order = torch.randperm(self.pages, generator=torch.Generator().manual_seed(seed + 1))
        table = torch.full((self.B, self.width + extra_columns), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n].int()
            at += n
        self.table, self.ldtable = table.cuda(), self.width + extra_columns
        self.lens = torch.tensor(list(lens), dtype=torch.int32, device="cuda")
        self.eight = cache == "e4m3"
        size = heads * page * D
        stride = size + gap
        kind = torch.uint8 if self.eight else TORCH[cache]
        self.ldpage = 2 * stride if both else stride
        if both:
            buf = torch.empty(self.pages * 2 * stride, dtype=kind, device="cuda")
            views = [buf, buf[stride:]]
        else:
            views = [torch.empty(self.pages * stride, dtype=kind, device="cuda") for _ in "kv"]
            buf = None
        self.buffers = [buf] if both else views
        self.pools = [v.as_strided((self.pages, heads, page, D), (self.ldpage, page * D, D, 1))
                      for v in views]
        for b in self.buffers:
            b.fill_(0x7F if self.eight else float("nan"))             # gaps
        for p in self.pools:
            v = torch.randn(p.shape, generator=g, device="cuda")
            if self.eight:
                p.copy_((v * 110).clamp(-448, 448).to(E4M3).view(torch.uint8))
            else:
                p.copy_(v)
        self.scales = [(0.005 + 0.01 * torch.rand(self.pages, heads, page, generator=g,
                                                  device="cuda")) if self.eight else None
                       for _ in "kv"]

    def args(self):
        """kcache .. lens, as the binding wants them."""
        return (self.pools[0], self.pools[1], self.scales[0], self.scales[1], self.pages, self.page,
                self.table, self.width, self.lens)

    def strides(self):
        return dict(ldpage=self.ldpage, ldtable=self.ldtable)

    def values(self, which):
        """The pool in binary64."""
        p = self.pools[which].contiguous()
        if not self.eight:
            return p.double().cpu().numpy()
        codes = p.view(E4M3).float().double().cpu().numpy()
        return codes * self.scales[which].double().cpu().numpy()[..., None]

    def places(self, b, lo, hi):
        """(pages, slots) of positions [lo, hi) of sequence b; page -1: not there."""
        n = min(max(self.lens_host[b], 0), self.width * self.page)
        j = np.arange(max(lo, 0), min(hi, n))
        t = self.table.cpu().numpy()
        pages = t[b, j // self.page].astype(np.int64)
        pages[(pages < 0) | (pages >= self.pages)] = -1
        return pages, j % self.page


def quantised(x: torch.Tensor):
    """Codes and scales of the rows of x (binary32, last axis), bit for bit: the scale and
    the quotient are products with rounded reciprocals."""
    x = x.float().cpu().numpy()
    with np.errstate(invalid="ignore"):
        top = np.where(np.isnan(x), 0, np.abs(x)).max(-1).astype(np.float32)
    scale = np.maximum(top, np.float32(LEAST)) * np.float32(np.float32(1) / np.float32(448))
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        inv = np.float32(1) / scale
        t = (x * inv[..., None]).astype(np.float32)
    nan = np.isnan(t)
    codes = torch.from_numpy(np.where(nan, 0, np.clip(t, -448, 448))).to(E4M3).view(torch.uint8)
    return torch.where(torch.from_numpy(nan), 0x7F, codes & 0xFF), torch.from_numpy(scale)
