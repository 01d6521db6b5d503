"""One mixture-of-experts layer around the tensor-parallel all-reduce.

serve(): R ranks' partial attention outputs are summed (ar_allreduce_n), added to
the residual stream and normalised to E4M3 with a scale per 128 elements
(ar_rmsnorm); every token's row goes to its top-K experts (ar_moe_route,
ar_moe_dispatch), through their two products (ar_matmul8), and back with its gate
weights (ar_moe_return).

train(): the same layer in bf16 with plain experts, forward and backward: the
norm with its rstd, the order, the return, and the gradients of all three
(ar_moe_return_grad, ar_moe_return without weights for the dispatch,
ar_rmsnorm_grad).

    python examples/moe_layer.py [--tokens 64] [--hidden 8192] [--experts 64] ...

runs both on cuda:0, checks them against plain torch and prints the errors and the
time of a serving step.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import all_reduce_reduction_gb300 as ar  # noqa: E402

EPS = 1e-6
TOP = 448.0


def blocks(n: int) -> int:
    return -(-n // ar.AR_SCALE_BLOCK)


def quantise(x: torch.Tensor, rows: int):
    """E4M3 codes of x (..., n, k) and their scales, one per `rows` x 128 block."""
    n, k = x.shape[-2:]
    b = ar.AR_SCALE_BLOCK
    full = torch.zeros(*x.shape[:-2], -(-n // rows) * rows, blocks(k) * b, device=x.device)
    full[..., :n, :k] = x
    cut = full.unflatten(-1, (-1, b)).unflatten(-3, (-1, rows))
    scale = cut.abs().amax((-3, -1)).clamp(min=2.0 ** -96) / TOP
    codes = (cut / scale[..., :, None, :, None]).to(torch.float8_e4m3fn)
    codes = codes.flatten(-2).flatten(-3, -2)[..., :n, :k]
    return codes.contiguous(), scale.contiguous()


def dequantise(codes: torch.Tensor, scale: torch.Tensor, rows: int) -> torch.Tensor:
    s = scale.repeat_interleave(ar.AR_SCALE_BLOCK, -1)[..., : codes.shape[-1]]
    if rows > 1:
        s = s.repeat_interleave(rows, -2)[..., : codes.shape[-2], :]
    return codes.float() * s


class Layer:
    """Weights and buffers of one layer, laid out once."""

    def __init__(self, tokens, hidden, inner, experts, top, ranks, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, scale=1.0):
            return torch.randn(*shape, generator=g, device="cuda") * scale
        self.T, self.H, self.I, self.E, self.K, self.R = tokens, hidden, inner, experts, top, ranks
        T, H, n = tokens, hidden, tokens * top
        self.gamma = (1 + 0.1 * normal(H)).bfloat16()
        self.router = normal(H, experts, scale=H ** -0.5)
        self.up = quantise(normal(experts, 2 * inner, H, scale=H ** -0.5), 128)
        self.down = quantise(normal(experts, H, inner, scale=inner ** -0.5), 128)
        self.partial = [normal(T, H, scale=ranks ** -0.5).bfloat16() for _ in range(ranks)]
        self.residual = normal(T, H).bfloat16()
        bf16, e4m3 = dict(dtype=torch.bfloat16, device="cuda"), dict(dtype=torch.float8_e4m3fn,
                                                                     device="cuda")
        self.attention = [torch.empty(T, H, **bf16) for _ in range(ranks)]
        self.total, self.out = torch.empty(T, H, **bf16), torch.empty(T, H, **bf16)
        self.x, self.xs = torch.empty(T, H, **e4m3), torch.empty(T, blocks(H), device="cuda")
        self.offsets = torch.empty(experts + 1, dtype=torch.int32, device="cuda")
        self.row_of = torch.empty(T, top, dtype=torch.int32, device="cuda")
        self.rows, self.rs = torch.zeros(n, H, **e4m3), torch.zeros(n, blocks(H), device="cuda")
        self.hidden = torch.zeros(n, 2 * inner, **bf16)
        self.y = torch.zeros(n, H, **bf16)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")   # of the products
        self.handle = ar.Handle(ranks, T * H, "bf16")

    def choose(self, normed: torch.Tensor):
        """The router's choices: expert ids and gate weights."""
        score, ids = torch.topk(normed @ self.router, self.K, dim=1)
        return ids, torch.softmax(score, 1).contiguous()

    def serve(self) -> torch.Tensor:
        T, H, K, n = self.T, self.H, self.K, self.T * self.K
        ar.ar_allreduce_n(self.handle.h, self.partial, self.attention, T * H)
        ar.ar_rmsnorm(self.attention[0], self.residual, self.gamma, EPS, self.total, self.x,
                      self.xs, None, T, H, "bf16", "e4m3")
        self.ids, self.w = self.choose(dequantise(self.x, self.xs, 1))
        ar.ar_moe_route(self.ids, T, K, self.E, self.offsets, self.row_of)
        ar.ar_moe_dispatch(self.x, self.xs, self.row_of, self.rows, self.rs, n, T, K, H, "e4m3")
        ar.ar_matmul8(self.rows, self.rs, *self.up, self.offsets, self.E, self.hidden, n,
                      2 * self.I, H, "bf16", status=self.status)
        gate, value = self.hidden.float().chunk(2, 1)
        act, act_scale = quantise(torch.nn.functional.silu(gate) * value, 1)
        ar.ar_matmul8(act, act_scale, *self.down, self.offsets, self.E, self.y, n, H, self.I,
                      "bf16", status=self.status)
        ar.ar_moe_return(self.y, n, self.row_of, self.w, self.out, T, K, H, "bf16")
        return self.out

    def check(self) -> None:
        """Raises if a product or the all-reduce gave up: the step's output is unfinished
        then.  Waits for the device, so a program calls it where it reads its results."""
        for what, status in (("ar_matmul8", int(self.status)),
                             ("ar_allreduce_n", ar.ar_status(self.handle.h))):
            if status != ar.AR_OK:
                raise ar.ArError(status, what)

    def serve_plain(self) -> torch.Tensor:
        """The same layer in plain torch, binary32, from the codes and choices of serve()."""
        x = dequantise(self.x, self.xs, 1)
        up, down = dequantise(*self.up, 128), dequantise(*self.down, 128)
        out = torch.zeros(self.T, self.H, device="cuda")
        for e in range(self.E):
            t, k = torch.nonzero(self.ids == e, as_tuple=True)
            if t.numel():
                gate, value = (x[t] @ up[e].t()).chunk(2, 1)
                act = torch.nn.functional.silu(gate) * value
                out.index_add_(0, t, self.w[t, k, None] * (act @ down[e].t()))
        return out

    def train(self):
        """Forward and backward of norm -> dispatch -> experts -> return in bf16.
        Returns the gradients of the input and of gamma, by this library and by
        torch's own differentiation in binary32."""
        T, H, K, n, E = self.T, self.H, self.K, self.T * self.K, self.E
        g = torch.Generator(device="cuda").manual_seed(1)
        x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
        d_out = torch.randn(T, H, generator=g, device="cuda").bfloat16()
        weight = [torch.randn(H, H, generator=g, device="cuda").bfloat16() * H ** -0.5
                  for _ in range(E)]
        normed, rstd = torch.empty_like(x), torch.empty(T, device="cuda")
        ar.ar_rmsnorm(x, None, self.gamma, EPS, None, normed, None, rstd, T, H, "bf16")
        ids, w = self.choose(normed.float())
        ar.ar_moe_route(ids, T, K, E, self.offsets, self.row_of)
        rows, y, out = torch.empty(n, H, dtype=x.dtype, device="cuda"), torch.empty(
            n, H, dtype=x.dtype, device="cuda"), torch.empty_like(x)
        ar.ar_moe_dispatch(normed, None, self.row_of, rows, None, n, T, K, H, "bf16")
        ends = self.offsets.tolist()
        for e in range(E):
            torch.matmul(rows[ends[e]:ends[e + 1]], weight[e], out=y[ends[e]:ends[e + 1]])
        ar.ar_moe_return(y, n, self.row_of, w, out, T, K, H, "bf16")

        d_y, d_w = torch.empty_like(y), torch.empty_like(w)
        ar.ar_moe_return_grad(d_out, y, n, self.row_of, w, d_y, d_w, T, K, H, "bf16")
        d_rows = torch.empty_like(rows)
        for e in range(E):
            torch.matmul(d_y[ends[e]:ends[e + 1]], weight[e].t(), out=d_rows[ends[e]:ends[e + 1]])
        d_normed, d_x = torch.empty_like(x), torch.empty_like(x)
        ar.ar_moe_return(d_rows, n, self.row_of, None, d_normed, T, K, H, "bf16")
        d_gamma = torch.empty(H, device="cuda")
        work = torch.empty(min(T, ar.AR_NORM_GRAD_ROWS) * H, device="cuda")
        ar.ar_rmsnorm_grad(d_normed, None, x, self.gamma, rstd, d_x, d_gamma, work,
                           4 * work.numel(), T, H, "bf16")

        px, pg, pw = (t.float().requires_grad_() for t in (x, self.gamma, w))
        plain = px * torch.rsqrt(px.square().mean(1, keepdim=True) + EPS) * pg
        result = torch.zeros(T, H, device="cuda")
        for e in range(E):
            t, k = torch.nonzero(ids == e, as_tuple=True)
            result = result.index_add(0, t, pw[t, k, None] * (plain[t] @ weight[e].float()))
        result.backward(d_out.float())
        return {"out": (out, result.detach()), "d_x": (d_x, px.grad), "d_gamma": (d_gamma, pg.grad),
                "d_w": (d_w, pw.grad)}

    def close(self) -> None:
        self.handle.close()


def off(got: torch.Tensor, want: torch.Tensor) -> float:
    """2-norm of the difference over the 2-norm of `want`."""
    return float((got.double() - want.double()).norm() / want.double().norm())


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, default in (("tokens", 64), ("hidden", 8192), ("inner", 1024), ("experts", 32),
                          ("top", 8), ("ranks", 8)):
        p.add_argument("--" + name, type=int, default=default)
    a = p.parse_args()
    torch.cuda.set_device(0)
    layer = Layer(a.tokens, a.hidden, a.inner, a.experts, a.top, a.ranks)
    out = layer.serve()
    layer.check()
    print("serving step against plain torch: %.2e off (the activations' E4M3 rounding between "
          "the products is in it)" % off(out, layer.serve_plain()))
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for _ in range(3):
        layer.serve()
    begin.record()
    for _ in range(20):
        layer.serve()
    end.record()
    end.synchronize()
    layer.check()
    print("serving step, %d tokens: %.1f us" % (a.tokens, begin.elapsed_time(end) / 20 * 1e3))
    for name, (got, want) in layer.train().items():
        print("training step, %s: %.2e off" % (name, off(got, want)))
    layer.close()


if __name__ == "__main__":
    main()
