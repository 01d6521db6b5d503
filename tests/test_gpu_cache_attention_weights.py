"""Small weights of ar_cache_attention on the GPU against the definition in binary64.

A position that takes nearly all of the weight and has values of zero leaves the output to the
others, whose weights are small: the error counts relative to what they make of the output.

Bound.  That of test_gpu_cache_attention.py, but for how a weight is held where keys and values
have two bytes or one: bf16 with 15 bits or more, binary16 and E4M3 with 12 bits or more where
the output is bf16, 14 where it is binary16, 16 where it is binary32; b bits are 2^-b of it:
  |out - want| <= 2 (e + chain + 2^-b) sum p|v| + half a unit of the output.
Weights here stay above 2^-43 of the largest."""
import numpy as np
import pytest
import torch

import all_reduce_reduction_gb300 as ar
from cache_helpers import E4M3, Cache
from gpu_helpers import need_gpu
from layer_helpers import TORCH, U, assert_within, f64, half

pytestmark = pytest.mark.gpu

BITS = {("bf16", "bf16"): 15, ("bf16", "e4m3"): 12, ("fp16", "fp16"): 14, ("fp16", "e4m3"): 14,
        ("fp32", "e4m3"): 16}
KINDS = [("bf16", "bf16"), ("bf16", "e4m3"), ("fp16", "fp16"), ("fp16", "e4m3"), ("fp32", "fp32"),
         ("fp32", "e4m3")]


def _positions(c, which, b, j):
    pages, slots = c.places(b, j, j + 1)
    return c.pools[which][int(pages[0]), :, int(slots[0])]


def _check(n, sinks, gap, dtype, cache, D=64, group=8, page=16, width=None, up=1.0):
    """One sequence of n positions: those in `sinks` score `gap`, all others 0; values of the
    first are 0, of the others between up / 2 and 3 up / 2."""
    need_gpu()
    c = Cache([n], 1, D, page, dtype, cache, seed=n)
    g = torch.Generator(device="cuda").manual_seed(n + 1)
    c.pools[0].zero_()
    v = 0.5 + torch.rand(c.pools[1].shape, generator=g, device="cuda")
    v[..., 5] = 1.0
    if c.eight:
        c.pools[1].copy_(v.to(E4M3).view(torch.uint8))
        c.scales[0].fill_(1.0)
        c.scales[1].fill_(up)
        key = int(torch.tensor(float(gap)).to(E4M3).view(torch.uint8))
    else:
        c.pools[1].copy_(v * up)
        key = gap
    for j in sinks:
        _positions(c, 0, 0, j)[:, 0] = key
        _positions(c, 1, 0, j).zero_()
    q = torch.zeros(1, group * D, device="cuda").to(TORCH[dtype])
    q.view(group, D)[:, 0] = 1.0
    args, kw = list(c.args()), c.strides()
    if width:
        table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
        table[:, :c.width] = c.table[:, :c.width]
        args[6], args[7], kw["ldtable"] = table, width, width
    out, lse = torch.full_like(q, float("nan")), torch.zeros(1, group, device="cuda")
    work = torch.full((ar.AR_CACHE_WORK_ROWS * (D + 2),), float("nan"), device="cuda")
    ar.ar_cache_attention(q, *args, 1.0, out, lse, work, 4 * work.numel(), 1, group, 1, D, dtype,
                          cache, **kw)
    torch.cuda.synchronize()
    pages, slots = c.places(0, 0, n)
    values = c.values(1)[pages, 0, slots]                             # n, D
    s = np.zeros(n)
    s[list(sinks)] = gap
    p = np.exp(s - s.max())
    p /= p.sum()
    want, size = p @ values, p @ np.abs(values)
    e = (D + 40) * U * gap + 8 * U + (n / 16 + 128) * U
    e += 2.0 ** -BITS[dtype, cache] if (dtype, cache) in BITS else 0
    bound = 2 * e * size + half(want, dtype) * (1 + 1e-6) + (2 * n + 2) * 2.0 ** -150
    assert_within(f64(out).reshape(group, D), np.tile(want, (group, 1)), np.tile(bound, (group, 1)),
                  "out")
    assert np.allclose(lse.double().cpu().numpy(), gap + np.log(np.exp(s - gap).sum()), atol=1e-4)


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("gap", [6, 8, 10, 12, 13, 14, 15, 16, 18, 20, 24, 28])
@pytest.mark.parametrize("sinks", [[0], [0, 16, 32, 48]], ids=len)
def test_one_position_and_one_in_each_group_of_warps(dtype, cache, gap, sinks):
    """A sequence that one CTA finishes (its table has room for no more) and one that is
    split over many."""
    up = 2.0 ** 10 if dtype == "fp16" else 1.0
    _check(4096, sinks, gap, dtype, cache, up=up)
    _check(4096, sinks, gap, dtype, cache, up=up, width=3000)


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("n", [2, 16, 17, 64, 65, 300])
def test_in_one_tile(dtype, cache, n):
    """The large weight among the 16 positions of the small ones, first and last."""
    for gap in (9, 14, 18, 26):
        for sink in (0, n - 1):
            _check(n, [sink], gap, dtype, cache, up=2.0 ** 12)


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("D,group", [(64, 1), (64, 16), (64, 32), (128, 8), (128, 16), (128, 32),
                                     (96, 8), (256, 8), (256, 16), (256, 32), (100, 8), (250, 3)])
def test_forms(dtype, cache, D, group):
    for gap in (15, 18):
        _check(1000, [3], gap, dtype, cache, D=D, group=group, up=2.0 ** 12)
        _check(1000, [3], gap, dtype, cache, D=D, group=group, page=10, up=2.0 ** 12, width=700)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_large_weights_of_tiny_scales(dtype):
    """E4M3: the others' scales are 2^-20 of the large weight's, or 2^20 times that."""
    for up in (2.0 ** -12, 2.0 ** 14):
        _check(500, [7], 12, dtype, "e4m3", up=up)
