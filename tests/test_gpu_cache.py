"""ar_cache_write and ar_cache_read on the GPU, bit for bit: 16- and 32-bit caches move
bits, E4M3 codes and scales are those of the stated products, a value read is
round(code * scale) with one binary32 product."""
import numpy as np
import pytest
import torch

import all_reduce_reduction_gb300 as ar
from cache_helpers import E4M3, Cache, quantised
from gpu_helpers import need_gpu
from layer_helpers import TORCH, placed, randn, untouched

pytestmark = pytest.mark.gpu


def _rows(seed, T, cols, dtype, pad, shift=0):
    return placed(randn(seed, T, cols).to(TORCH[dtype]).cuda(), pad, shift)


def _targets(c, new, T):
    """(row, page, slot) of every row with a place; new None: one a sequence."""
    out, at = [], 0
    for b in range(c.B):
        m = 1 if new is None else new[b]
        n = min(max(c.lens_host[b], 0), c.width * c.page)
        for i in range(m):
            j = n - m + i
            if j >= 0:
                (p,), (s,) = c.places(b, j, j + 1)
                if p >= 0:
                    out.append((at + i, int(p), int(s)))
        at += m
    return [r for r in out if r[0] < T]


def _offsets(new):
    return None if new is None else torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32,
                                                 device="cuda")


def _bits(t):
    return t.view(torch.uint8) if t.dtype == E4M3 else t.view(
        {1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def _check(lens, new, heads, D, page, dtype, cache, pad=0, shift=0, extra_rows=0, **kw):
    need_gpu()
    c = Cache(lens, heads, D, page, dtype, cache, **kw)
    T = (c.B if new is None else sum(new)) + extra_rows
    cols = heads * D
    k, kbuf = _rows(1, T, cols, dtype, pad, shift)
    v, vbuf = _rows(2, T, cols, dtype, pad, shift)
    off = _offsets(new)
    want = [b.clone() for b in c.buffers]
    ref = Cache.__new__(Cache)
    ref.__dict__.update(c.__dict__)
    # the same views of the copies
    ref.pools = [w.as_strided(p.shape, p.stride(), p.storage_offset())
                 for w, p in zip(want * (2 // len(want)), c.pools)]
    scales = [None if s is None else s.clone() for s in c.scales]
    targets = _targets(c, new, T)
    for pool, scale, x in zip(ref.pools, scales, (k, v)):
        x = x.reshape(T, heads, D)
        if c.eight:
            codes, s = quantised(x)
            codes, s = codes.cuda(), s.cuda()
        for row, p, slot in targets:
            if c.eight:
                pool[p, :, slot] = codes[row]
                scale[p, :, slot] = s[row]
            else:
                pool[p, :, slot] = x[row]
    ar.ar_cache_write(k, v, *c.args(), off, T, c.B, heads, D, dtype, cache, ldk=cols + pad,
                      ldv=cols + pad, **c.strides())
    torch.cuda.synchronize()
    for got, w in zip(c.buffers, want):
        assert torch.equal(_bits(got), _bits(w))
    if c.eight:
        for got, w in zip(c.scales, scales):
            assert torch.equal(got, w)
    # back, into rows of NaN: those without a place stay
    rk, rkbuf = placed(torch.full((T, cols), float("nan"), device="cuda").to(TORCH[dtype]), pad,
                       shift)
    rv, rvbuf = placed(torch.full((T, cols), float("nan"), device="cuda").to(TORCH[dtype]), pad,
                       shift)
    ar.ar_cache_read(*c.args(), off, rk, rv, T, c.B, heads, D, dtype, cache, ldk=cols + pad,
                     ldv=cols + pad, **c.strides())
    torch.cuda.synchronize()
    for got, buf, pool, scale in ((rk, rkbuf, c.pools[0], c.scales[0]),
                                  (rv, rvbuf, c.pools[1], c.scales[1])):
        assert untouched(buf, T, cols, pad, shift)
        expect = torch.full((T, heads, D), float("nan"), device="cuda").to(TORCH[dtype])
        for row, p, slot in targets:
            cells = pool[p, :, slot]
            if c.eight:
                cells = cells.contiguous().view(E4M3).float() * scale[p, :, slot][:, None]
            expect[row] = cells.to(TORCH[dtype])
        expect = expect.reshape(T, cols)
        same = _bits(got.contiguous()) == _bits(expect)
        assert bool((same | (torch.isnan(got) & torch.isnan(expect))).all())


KINDS = [("bf16", "bf16"), ("bf16", "e4m3"), ("fp16", "fp16"), ("fp16", "e4m3"), ("fp32", "fp32"),
         ("fp32", "e4m3")]


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("D", [1, 5, 8, 16, 33, 64, 80, 96, 100, 128, 192, 200, 255, 256])
def test_head_sizes(dtype, cache, D):
    _check([5, 1, 40, 17], None, 3, D, 16, dtype, cache, seed=D)
    _check([9, 4, 30], [3, 4, 17], 2, D, 7, dtype, cache, seed=D + 1, pad=D % 2 * 8)


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("lens,new", [
    ([1], None), ([0, 1, 2], None), ([0], [0]), ([0, 0, 5], [0, 0, 5]), ([3, 0, 9], [3, 0, 1]),
    ([100, 3], [64, 3]), ([2, 4], [5, 4]), ([300], [300]), ([-4, 7], [2, 2]), ([70] * 40, None),
    ([65] * 9, [33] * 9)], ids=str)
def test_sequences(dtype, cache, lens, new):
    """Empty ones, lengths below the new rows, one token, rows across pages."""
    _check(lens, new, 4, 64, 16, dtype, cache, seed=len(lens))
    _check(lens, new, 1, 20, 5, dtype, cache, seed=3, extra_rows=0 if new is None else 3)


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("pad,shift,gap,both", [
    (0, 0, 0, True), (16, 0, 32, False), (3, 0, 0, False), (0, 1, 0, False), (8, 8, 5, True),
    (0, 0, 1, False), (5, 3, 7, True)])
def test_strides_and_alignment(dtype, cache, pad, shift, gap, both):
    _check([20, 33, 8], [5, 30, 8], 2, 64, 16, dtype, cache, pad=pad, shift=shift, gap=gap,
           both=both, extra_columns=3, seed=pad)


@pytest.mark.parametrize("heads,page", [(1, 1), (24, 3), (130, 2), (1024, 1), (6, 100)])
def test_heads_and_pages(heads, page):
    """Up to several CTAs a row, and pages of one slot."""
    _check([5, 9], [5, 4], heads, 128, page, "bf16", "e4m3")
    _check([5, 9], None, heads, 16, page, "fp32", "fp32")
    _check([5, 9], [2, 4], heads, 36, page, "fp16", "e4m3")


def test_many_rows():
    _check([5000, 0, 700], [4100, 0, 700], 8, 128, 64, "bf16", "e4m3")
    _check([2000, 1500], [2000, 1111], 3, 80, 16, "fp16", "fp16")


def _spoiled(**kw):
    c = Cache([30, 40, 12], 2, 64, 8, "bf16", "e4m3", **kw)
    return c


def test_pages_outside_the_pool_are_skipped():
    """Words of the table below 0 and past the pool, lengths below 0 and past the table."""
    need_gpu()
    c = _spoiled(spare=3)
    c.table[0, 1], c.table[1, 0], c.table[1, 4] = c.pages, -2 ** 31, 2 ** 31 - 1
    c.lens_host = [30, 2 ** 31 - 1, -5]
    c.lens.copy_(torch.tensor(c.lens_host, dtype=torch.int32))
    new = [20, 39, 3]
    before = [b.clone() for b in c.buffers]
    k, v = (randn(s, 62, 128).bfloat16().cuda() for s in (1, 2))
    ar.ar_cache_write(k, v, *c.args(), _offsets(new), 62, 3, 2, 64, "bf16", "e4m3", **c.strides())
    torch.cuda.synchronize()
    targets = _targets(c, new, 62)
    assert 0 < len(targets) < 59
    codes, scale = quantised(k.view(62, 2, 64))
    want = before[0].view(c.pages, 2, 8, 64)
    for row, p, s in targets:
        want[p, :, s] = codes[row].cuda()
        assert torch.equal(c.scales[0][p, :, s].cpu(), scale[row])
    assert torch.equal(c.buffers[0], want.view(-1))
    out = [torch.full((62, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    ar.ar_cache_read(*c.args(), _offsets(new), *out, 62, 3, 2, 64, "bf16", "e4m3", **c.strides())
    there = torch.zeros(62, dtype=torch.bool, device="cuda")
    there[torch.tensor([t[0] for t in targets], device="cuda")] = True
    assert bool((out[0][~there] == 7).all()) and bool((out[1][~there] == 7).all())
    assert not bool((out[0][there] == 7).all(1).any())


@pytest.mark.parametrize("offsets", [[5, 2, 9, 4], [-3, 4, 4, 100], [0, 0, 0, 0], [60, 70, 80, 90],
                                     [-2 ** 31, 0, 0, 2 ** 31 - 1]], ids=str)
def test_offsets_that_are_no_order(offsets):
    """Whatever they hold, only places of the sequences' own pages are written."""
    need_gpu()
    c = _spoiled()
    before = [b.clone() for b in c.buffers]
    k, v = (randn(s, 50, 128).bfloat16().cuda() for s in (1, 2))
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    ar.ar_cache_write(k, v, *c.args(), off, 50, 3, 2, 64, "bf16", "e4m3", **c.strides())
    torch.cuda.synchronize()
    used = c.table[c.table >= 0].long()
    free = torch.ones(c.pages, dtype=torch.bool, device="cuda")
    free[used] = False
    for now, was in zip(c.buffers, before):
        assert torch.equal(now.view(c.pages, -1)[free], was.view(c.pages, -1)[free])


def test_special_values():
    """Zeros, the smallest and largest numbers, infinities and NaN in rows of their own."""
    need_gpu()
    D, heads = 64, 1
    rows = torch.zeros(8, D)
    rows[1] = 2.0 ** -126
    rows[2] = 3e38
    rows[3, 5] = float("inf")
    rows[4, 7] = float("nan")
    rows[5] = float("nan")
    rows[6] = torch.linspace(-1, 1, D)
    rows[7, 0] = -2.0 ** -100
    for dtype in ("fp32", "bf16"):
        x = rows.to(TORCH[dtype]).cuda()
        c = Cache([8], heads, D, 8, dtype, "e4m3")
        ar.ar_cache_write(x, x, *c.args(), _offsets([8]), 8, 1, heads, D, dtype, "e4m3")
        codes, scale = quantised(x)
        page = int(c.table[0, 0])
        got = c.pools[0][page, 0]
        same = (got.cpu() == codes) | ((got.cpu() & 0x7F == 0x7F) & (codes & 0x7F == 0x7F))
        assert bool(same.all())
        s = c.scales[0][page, 0].cpu()
        assert torch.equal(s, scale)


def test_in_a_graph_as_the_sequences_grow():
    """One capture serves every step: lengths and pages are read on the device."""
    need_gpu()
    c = Cache([30, 30, 30], 2, 128, 8, "bf16", "e4m3", width=4)
    k, v = (torch.zeros(3, 256, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    rk, rv = torch.zeros_like(k), torch.zeros_like(v)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        ar.ar_cache_write(k, v, *c.args(), None, 3, 3, 2, 128, "bf16", "e4m3", stream=s)
        ar.ar_cache_read(*c.args(), None, rk, rv, 3, 3, 2, 128, "bf16", "e4m3", stream=s)
    for step, lens in enumerate(([1, 9, 30], [2, 10, 31], [3, 0, 32])):
        c.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        x = randn(step, 2, 3, 256).bfloat16().cuda()
        k.copy_(x[0])
        v.copy_(x[1])
        rk.fill_(9)
        g.replay()
        torch.cuda.synchronize()
        codes, scale = quantised(k.view(3, 2, 128))
        want = (codes.view(E4M3).float() * scale[..., None]).bfloat16().view(3, 256).cuda()
        there = torch.tensor([n > 0 for n in lens], device="cuda")
        assert torch.equal(rk[there], want[there])
        assert bool((rk[~there] == 9).all())


def test_zero_rows_and_other_streams():
    need_gpu()
    c = Cache([4], 1, 64, 4, "fp16", "fp16")
    before = c.buffers[0].clone()
    ar.ar_cache_write(None, None, *c.args(), _offsets([0]), 0, 1, 1, 64, "fp16")
    s = torch.cuda.Stream()
    x = torch.ones(1, 64, dtype=torch.float16, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda.current_stream().synchronize()
    assert torch.equal(c.buffers[0], before)
    with torch.cuda.stream(s):
        ar.ar_cache_write(x, x, *c.args(), None, 1, 1, 1, 64, "fp16")
    s.synchronize()
    assert bool((c.pools[0][int(c.table[0, 0]), 0, 3] == 1).all())
