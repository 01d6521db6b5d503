"""Caches and weights past 4 GiB: byte offsets that do not fit 32 bits."""
import math

import pytest
import torch

import all_reduce_reduction_gb300 as ar
from gpu_helpers import need_gpu
from layer_helpers import f64

pytestmark = pytest.mark.gpu

HEADS, D, PAGE = 8, 128, 64
MARK = (1 << 32) // (HEADS * D * PAGE)                  # pages of 4 GiB of codes


@pytest.mark.parametrize("cache", ["e4m3", "bf16", "fp32"])
def test_cache(cache):
    """Pages on both sides of the mark, written, read and attended to."""
    need_gpu()
    size = {"e4m3": 1, "bf16": 2, "fp32": 4}[cache]
    mark = MARK // size
    pages = mark + 40
    dtype = "fp32" if cache == "fp32" else "bf16"
    t = torch.float32 if cache == "fp32" else torch.bfloat16
    kind = torch.uint8 if cache == "e4m3" else t
    pools = [torch.zeros(pages, HEADS, PAGE, D, dtype=kind, device="cuda") for _ in "kv"]
    scales = [torch.zeros(pages, HEADS, PAGE, device="cuda") if cache == "e4m3" else None
              for _ in "kv"]
    order = [0, mark - 1, mark, mark + 1, pages - 1, mark + 7]
    table = torch.tensor([order], dtype=torch.int32, device="cuda")
    n = PAGE * len(order) - 11
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    k, v, q = (torch.randn(rows, HEADS * D, generator=g, device="cuda").to(t)
               for rows in (n, n, 1))
    args = (*pools, *scales, pages, PAGE, table, len(order), lens)
    ar.ar_cache_write(k, v, *args, offsets, n, 1, HEADS, D, dtype, cache)
    back = [torch.zeros_like(k) for _ in "kv"]
    ar.ar_cache_read(*args, offsets, *back, n, 1, HEADS, D, dtype, cache)
    for got, want in zip(back, (k, v)):
        if cache != "e4m3":
            assert torch.equal(got, want)
        else:
            top = want.float().view(n, HEADS, D).abs().amax(2, keepdim=True)
            err = (got.float() - want.float()).view(n, HEADS, D).abs()
            # half a step, 2^-4, a bf16 rounding and the scale's two; near zero 2^-10 of 448
            assert bool((err <= (2.0 ** -4 + 2.0 ** -8) * want.float().view(n, HEADS, D).abs()
                         + 2.0 ** -16 * top).all())
    # the first pages alone hold something
    assert not bool(pools[0][1].any()) and not bool(pools[1][mark - 2].any())
    out, lse = torch.zeros_like(q), torch.zeros(1, HEADS, device="cuda")
    work = torch.zeros(ar.AR_CACHE_WORK_ROWS * (D + 2), device="cuda")
    ar.ar_cache_attention(q, *args, D ** -0.5, out, lse, work, 4 * work.numel(), 1, HEADS, HEADS, D,
                          dtype, cache)
    # from what was read back, whose roundings to bf16 (2^-9 of a value) the cache in 8
    # bits does not have: they move a score by 2^-9 of sum |q||k| / sqrt(D) at most, its
    # weight by e times that, and a value by 2^-9
    kk, vv = (torch.from_numpy(f64(x)).view(n, HEADS, D) for x in back)
    qq = torch.from_numpy(f64(q)).view(HEADS, D)
    s = torch.einsum("hd,nhd->hn", qq, kk) / math.sqrt(D)
    p = torch.softmax(s, 1)
    want = torch.einsum("hn,nhd->hd", p, vv)
    size_of = torch.einsum("hn,nhd->hd", p, vv.abs())
    most = torch.einsum("hd,nhd->hn", qq.abs(), kk.abs()).amax(1)[:, None] / math.sqrt(D)
    rel = (2.0 ** -9 * (2.8 * most + 1) if cache == "e4m3" else 0) + 2.0 ** -15 + \
        300 * 2.0 ** -24 * (most + 1)
    bound = rel * size_of + (2.0 ** -24 if cache == "fp32" else 2.0 ** -8) * want.abs()
    got = torch.from_numpy(f64(out)).view(HEADS, D)
    assert bool(((got - want).abs() <= bound).all())


def test_expert_weights():
    """Experts on both sides of 4 GiB in each of the two matrices."""
    need_gpu()
    H, F, T, K = 4096, 4096, 2, 3
    E = (1 << 32) // (H * F) + 4                        # down: past 4 GiB; up: past 8
    up = torch.zeros(E, 2 * F, H, dtype=torch.uint8, device="cuda")
    down = torch.zeros(E, H, F, dtype=torch.uint8, device="cuda")
    ids = torch.tensor([[0, E // 2, E - 1], [E - 4, E // 2 + 1, E - 2]], dtype=torch.int32,
                       device="cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    for e in ids.flatten().tolist():
        for w in (up, down):
            x = torch.randn(w.shape[1:], generator=g, device="cuda").clamp(-4, 4) * 100
            w[e] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    us = torch.full((E, 2 * F // 128, H // 128), H ** -0.5 / 100, device="cuda")
    ds = torch.full((E, H // 128, F // 128), F ** -0.5 / 100, device="cuda")
    x, w = torch.randn(T, H, generator=g, device="cuda"), torch.rand(T, K, generator=g,
                                                                     device="cuda")
    out = torch.zeros(T, H, device="cuda")
    work = torch.zeros(T * K * (F + 128), device="cuda")
    ar.ar_moe_layer(x, ids, w, up, us, down, ds, out, work, 4 * work.numel(), T, K, E, H, F, "fp32")
    want, size = torch.zeros(T, H, dtype=torch.float64, device="cuda"), 0.0
    for t in range(T):
        for k in range(K):
            e = int(ids[t, k])
            w1 = up[e].view(torch.float8_e4m3fn).float().double() * us[e, 0, 0].double()
            w2 = down[e].view(torch.float8_e4m3fn).float().double() * ds[e, 0, 0].double()
            gate, value = (w1 @ x[t].double()).chunk(2)
            act = gate * torch.sigmoid(gate) * value
            want[t] += w[t, k].double() * (w2 @ act)
            size = max(size, float((w2.abs() @ act.abs()).max()))
    # 2^-21 for each of x and h, and some hundred units of 2^-24 for the sums; a g or a u
    # that is off moves h by as much of sum |up||x|, 64 times the square root's size at most
    assert float((out.double() - want).abs().max()) <= K * size * 64 * 2.0 ** -19
