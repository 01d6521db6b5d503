"""One decode step of a tensor-parallel mixture-of-experts layer over R virtual ranks.

Every rank has a share of the attention heads, with its own paged cache, and a share of
the experts.  A step takes one new token of every sequence through the layer:

    new keys and values into each rank's cache          ar_cache_write
    attention over it                                   ar_cache_attention
    the ranks' partial projections summed               ar_allreduce_n
    residual and norm                                   ar_rmsnorm
    each rank's experts for the tokens that chose them  ar_moe_layer
    the ranks' partial results summed                   ar_allreduce_n

The prompts' keys and values are written in one call before (a ragged batch), in E4M3 or
as they are.  The step is captured in a CUDA graph once; lengths, pages and choices are
read on the device, so the same graph serves every step.

    python examples/decode_layer.py [--sequences 16] [--context 2000] [--cache e4m3] ...

runs some steps on cuda:0, checks each against plain torch and prints the errors and the
time of a step.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import all_reduce_reduction_gb300 as ar  # noqa: E402
from moe_layer import EPS, dequantise, off, quantise  # noqa: E402

E4M3 = torch.float8_e4m3fn


class Cache:
    """One rank's pages, filled as the sequences grow."""

    def __init__(self, pages, heads, dim, page, kind):
        self.heads, self.dim, self.page, self.pages = heads, dim, page, pages
        self.kind = kind
        dtype = E4M3 if kind == "e4m3" else torch.bfloat16
        self.k, self.v = (torch.zeros(pages, heads, page, dim, dtype=dtype, device="cuda")
                          for _ in "kv")
        self.ks, self.vs = (torch.zeros(pages, heads, page, device="cuda")
                            if kind == "e4m3" else None for _ in "kv")

    def values(self, which, table, n):
        """Positions [0, n) of a sequence in binary32: n, heads, dim."""
        pool, scale = (self.k, self.ks) if which == "k" else (self.v, self.vs)
        j = torch.arange(n, device="cuda")
        at, slot = table[j // self.page].long(), j % self.page
        if scale is None:
            return pool[at, :, slot].float()
        codes = pool.view(torch.uint8)[at, :, slot].view(E4M3)
        return codes.float() * scale[at, :, slot][..., None]


class Decoder:
    def __init__(self, sequences, longest, hidden, heads, kv_heads, dim, page, inner, experts, top,
                 ranks, cache="e4m3", seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, scale=1.0):
            return torch.randn(*shape, generator=g, device="cuda") * scale
        self.B, self.H, self.R, self.K, self.E, self.F = (sequences, hidden, ranks, top, experts,
                                                          inner)
        self.q_heads, self.kv, self.D = heads // ranks, kv_heads // ranks, dim
        self.each = experts // ranks                             # experts of a rank
        B, H, R = sequences, hidden, ranks
        width = -(-longest // page)
        self.width = width
        order = torch.randperm(B * width, generator=g, device="cuda").int()
        self.table = order.view(B, width).contiguous()
        self.caches = [Cache(B * width, self.kv, dim, page, cache) for _ in range(R)]
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.columns = (self.q_heads + 2 * self.kv) * dim        # of a rank's first product
        self.qkv = [normal(H, self.columns, scale=H ** -0.5).bfloat16() for _ in range(R)]
        self.o = [normal(self.q_heads * dim, H, scale=H ** -0.5).bfloat16() for _ in range(R)]
        self.gamma = (1 + 0.1 * normal(H)).bfloat16()
        self.router = normal(H, experts, scale=H ** -0.5)
        self.up = [quantise(normal(self.each, 2 * inner, H, scale=H ** -0.5), 128)
                   for _ in range(R)]
        self.down = [quantise(normal(self.each, H, inner, scale=inner ** -0.5), 128)
                     for _ in range(R)]
        # buffers
        bf16 = dict(dtype=torch.bfloat16, device="cuda")
        self.x = torch.zeros(B, H, **bf16)                       # the tokens of this step
        self.first = [torch.zeros(B, self.columns, **bf16) for _ in range(R)]
        self.mixed = [torch.zeros(B, self.q_heads * dim, **bf16) for _ in range(R)]
        self.partial = [torch.zeros(B, H, **bf16) for _ in range(R)]
        self.summed = [torch.zeros(B, H, **bf16) for _ in range(R)]
        self.total, self.normed = torch.zeros(B, H, **bf16), torch.zeros(B, H, **bf16)
        self.expert = [torch.zeros(B, H, **bf16) for _ in range(R)]
        self.out = [torch.zeros(B, H, **bf16) for _ in range(R)]
        self.local = torch.zeros(B, top, dtype=torch.int64, device="cuda")
        # a workspace serves every rank here: their calls run one after the other
        self.work = torch.zeros(ar.AR_CACHE_WORK_ROWS * (dim + 2), device="cuda")
        self.moe_work = torch.zeros(B * top * (inner + 128), device="cuda")
        self.handle = ar.Handle(R, B * H, "bf16")

    def _cache_args(self, c):
        return (c.k, c.v, c.ks, c.vs, c.pages, c.page, self.table, self.width, self.lens)

    def _slices(self, first):
        """q, k and v of a rank's first product: columns of one buffer."""
        q, kv = self.q_heads * self.D, self.kv * self.D
        return first[:, :q], first[:, q:q + kv], first[:, q + kv:]

    def prompt(self, tokens, lengths):
        """The prompts' keys and values into the caches: rows of all sequences in one call."""
        offsets = torch.tensor([0] + lengths, device="cuda").cumsum(0).int()
        self.lens.copy_(torch.tensor(lengths, dtype=torch.int32))
        T = tokens.shape[0]
        self.prompt_rows = []
        for r, c in enumerate(self.caches):
            first = tokens @ self.qkv[r]
            _, k, v = self._slices(first)
            ar.ar_cache_write(k, v, *self._cache_args(c), offsets, T, self.B, self.kv, self.D,
                              "bf16", c.kind, ldk=self.columns, ldv=self.columns)
            self.prompt_rows.append((k, v, offsets))

    def step(self):
        B, H, K = self.B, self.H, self.K
        self.lens += 1                                           # counts the new token
        for r, c in enumerate(self.caches):
            torch.matmul(self.x, self.qkv[r], out=self.first[r])
            q, k, v = self._slices(self.first[r])
            ar.ar_cache_write(k, v, *self._cache_args(c), None, B, B, self.kv, self.D, "bf16",
                              c.kind, ldk=self.columns, ldv=self.columns)
            ar.ar_cache_attention(q, *self._cache_args(c), self.D ** -0.5, self.mixed[r], None,
                                  self.work, 4 * self.work.numel(), B, self.q_heads, self.kv,
                                  self.D, "bf16", c.kind, ldq=self.columns)
            torch.matmul(self.mixed[r], self.o[r], out=self.partial[r])
        ar.ar_allreduce_n(self.handle.h, self.partial, self.summed, B * H)
        ar.ar_rmsnorm(self.summed[0], self.x, self.gamma, EPS, self.total, self.normed, None, None,
                      B, H, "bf16")
        score, self.ids = torch.topk(self.normed.float() @ self.router, K, dim=1)
        self.w = torch.softmax(score, 1)
        for r in range(self.R):
            # a rank's experts are [0, each) to it; the others' ids fall outside
            torch.sub(self.ids, r * self.each, out=self.local)
            ar.ar_moe_layer(self.normed, self.local, self.w, *self.up[r], *self.down[r],
                            self.expert[r], self.moe_work, 4 * self.moe_work.numel(), B, K,
                            self.each, H, self.F, "bf16")
        ar.ar_allreduce_n(self.handle.h, self.expert, self.out, B * H)
        return self.out[0]

    def plain(self):
        """The step that was just made in plain torch, binary32, over the caches as they are:
        (attention's projections summed, the layer's output for the choices made)."""
        B, group = self.B, self.q_heads // self.kv
        lens = self.lens.tolist()
        total = torch.zeros(B, self.H, device="cuda")
        for r, c in enumerate(self.caches):
            q = self._slices(self.first[r])[0].float().view(B, self.kv, group, self.D)
            mixed = torch.zeros(B, self.kv, group, self.D, device="cuda")
            for b, n in enumerate(lens):
                k, v = c.values("k", self.table[b], n), c.values("v", self.table[b], n)
                s = torch.einsum("hgd,nhd->hgn", q[b], k) * self.D ** -0.5
                mixed[b] = torch.einsum("hgn,nhd->hgd", torch.softmax(s, 2), v)
            total += mixed.view(B, -1) @ self.o[r].float()
        x = self.normed.float()
        out = torch.zeros(B, self.H, device="cuda")
        for e in range(self.E):
            t, k = torch.nonzero(self.ids == e, as_tuple=True)
            if t.numel():
                up, down = ((w[e % self.each], s[e % self.each]) for w, s in
                            (self.up[e // self.each], self.down[e // self.each]))
                gate, value = (x[t] @ dequantise(*up, 128).t()).chunk(2, 1)
                act = torch.nn.functional.silu(gate) * value
                out.index_add_(0, t, self.w[t, k, None] * (act @ dequantise(*down, 128).t()))
        return total, out

    def captured(self):
        """The step as a graph: replay() makes the next one."""
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        kept = self.lens.clone()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            self.step()                                          # warm-up
            stream.synchronize()
            self.lens.copy_(kept)
            with torch.cuda.graph(graph, stream=stream):
                self.step()
        torch.cuda.current_stream().wait_stream(stream)
        return graph

    def check(self):
        status = ar.ar_status(self.handle.h)
        if status != ar.AR_OK:
            raise ar.ArError(status, "ar_allreduce_n")

    def close(self):
        self.handle.close()


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, default in (("sequences", 16), ("context", 2000), ("hidden", 8192), ("heads", 64),
                          ("kv-heads", 8), ("dim", 128), ("page", 64), ("inner", 1024),
                          ("experts", 64), ("top", 8), ("ranks", 8), ("steps", 3)):
        p.add_argument("--" + name, type=int, default=default)
    p.add_argument("--cache", choices=("e4m3", "bf16"), default="e4m3")
    a = p.parse_args()
    torch.cuda.set_device(0)
    d = Decoder(a.sequences, a.context + 200, a.hidden, a.heads, a.kv_heads, a.dim, a.page, a.inner,
                a.experts, a.top, a.ranks, a.cache)
    g = torch.Generator(device="cuda").manual_seed(1)
    lengths = [max(1, a.context * (b + 1) // a.sequences) for b in range(a.sequences)]
    d.prompt(torch.randn(sum(lengths), a.hidden, generator=g, device="cuda").bfloat16(), lengths)
    graph = d.captured()
    for i in range(a.steps):
        d.x.copy_(torch.randn(a.sequences, a.hidden, generator=g, device="cuda"))
        graph.replay()
        d.check()
        attention, out = d.plain()
        print("step %d against plain torch: attention %.2e off, layer %.2e off"
              % (i, off(d.summed[0], attention), off(d.out[0], out)))
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(20):
        graph.replay()
    end.record()
    end.synchronize()
    d.check()
    print("decode step, %d sequences, %d ranks one after the other: %.1f us"
          % (a.sequences, a.ranks, begin.elapsed_time(end) / 20 * 1e3))
    d.close()


if __name__ == "__main__":
    main()
