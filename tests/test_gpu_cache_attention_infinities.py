"""Infinities and NaN among the values of a sequence: what the definition makes of them, in
every form of ar_cache_attention.  A position's weight is positive, however small: an infinity
remains one, two of opposite signs give NaN, and no other column changes."""
import math

import pytest
import torch

import all_reduce_reduction_gb300 as ar
from cache_helpers import Cache
from gpu_helpers import need_gpu
from layer_helpers import TORCH, randn

pytestmark = pytest.mark.gpu

INF, NAN = math.inf, math.nan


def _check(dtype, n, group, D, page=16, gap=0, width=None, low=0.0, window=0, spoils=None):
    need_gpu()
    c = Cache([n, 40], 1, D, page, dtype, dtype, gap=gap, seed=D)

    def element(which, j, d):
        pages, slots = c.places(0, j, j + 1)
        return c.pools[which][int(pages[0]), 0, int(slots[0])][d:d + 1]
    if low:                               # a position of far less weight than the others
        c.pools[0][..., 0] = 0.0
        element(0, n // 2, 0).fill_(-low)
    args, kw = list(c.args()), c.strides()
    if width:
        table = torch.full((2, width), -1, dtype=torch.int32, device="cuda")
        table[:, :c.width] = c.table[:, :c.width]
        args[6], args[7], kw["ldtable"] = table, width, width
    q = randn(3, 2, group * D).to(TORCH[dtype]).cuda()
    q.view(2, group, D)[:, :, 0] = D ** 0.5 if low else 0.5
    if low:
        q.view(2, group, D)[:, :, 1:] *= 0.1
    work = torch.full((ar.AR_CACHE_WORK_ROWS * (D + 2),), NAN, device="cuda")

    def call():
        out, lse = torch.zeros_like(q), torch.zeros(2, group, device="cuda")
        ar.ar_cache_attention(q, *args, D ** -0.5, out, lse, work, 4 * work.numel(), 2, group, 1,
                              D, dtype, window=window, **kw)
        torch.cuda.synchronize()
        return out.view(2, group, D), lse
    clean, clean_lse = call()
    last = n - 1
    spoils = spoils or [(last, 1, INF, INF), (last, 2, -INF, -INF), (n // 2, 3, INF, INF),
                        (n // 2, 4, -INF, -INF), (n // 2, 5, NAN, NAN)]
    want = clean.clone()
    for j, d, value, result in spoils:
        element(1, j, d).fill_(value)
        want[0, :, d] = result
    if not low:
        element(1, n // 2, 6).fill_(INF)
        element(1, last, 6).fill_(-INF)
        want[0, :, 6] = NAN if n // 2 != last else -INF
    out, lse = call()
    assert torch.equal(torch.nan_to_num(out, nan=77), torch.nan_to_num(want, nan=77))
    assert torch.equal(lse, clean_lse)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n", [1, 2, 16, 17, 70, 300, 3000])
def test_lengths(dtype, n):
    _check(dtype, n, 8, 64)
    _check(dtype, n, 8, 64, width=3000)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("group,D,page,gap", [
    (1, 64, 16, 0), (16, 64, 16, 0), (32, 64, 16, 0), (8, 128, 16, 0), (16, 128, 10, 0),
    (32, 128, 16, 0), (8, 256, 16, 0), (16, 256, 16, 0), (32, 256, 7, 0), (8, 80, 16, 0),
    (8, 100, 16, 0), (4, 64, 16, 1), (3, 7, 5, 0)])
def test_forms_and_alignments(dtype, group, D, page, gap):
    _check(dtype, 500, group, D, page=page, gap=gap)
    _check(dtype, 500, group, D, page=page, gap=gap, width=2000, window=400)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("low", [8.0, 15.0, 16.0, 17.5, 20.0, 25.0, 40.0])
def test_of_little_weight(dtype, low):
    """exp(-40) of the others' weight is 2^-58 of it."""
    for n in (10, 64, 1000):
        _check(dtype, n, 8, 64, low=low)
        _check(dtype, n, 4, 128, low=low, width=2000)
