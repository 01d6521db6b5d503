"""ar_rmsnorm and its gradient on the GPU against the definitions in binary64.

Bounds.  v = x + res carries one rounding.  The sum of squares is a sum of at
most 64 sequential adds and two trees of depth 5 per thread (relative error at
most 80 u, all terms are positive); mean, eps, root and reciprocal add four
roundings, and half of the sum's error reaches r.  y adds two products.  So y
is within 64 u |y| of the exact value before its rounding, for H <= 65536."""
import numpy as np
import pytest
import torch

import all_reduce_reduction_gb300 as ar
from gpu_helpers import need_gpu
from layer_helpers import (LEAST, TORCH, U, assert_within, e4m3_step, f64, half, placed, randn,
                           untouched)

pytestmark = pytest.mark.gpu
EPS = 1e-5


def _inputs(T, H, dtype, seed):
    x = randn(seed, T, H).to(TORCH[dtype])
    res = (randn(seed + 1, T, H) * 8).to(TORCH[dtype])
    g = (1 + 0.2 * randn(seed + 2, H)).to(TORCH[dtype])
    return x, res, g


def _forward64(x, res, g, eps=EPS):
    v = f64(x) + (f64(res) if res is not None else 0.0)
    r = 1.0 / np.sqrt((v * v).mean(1) + eps)
    return v, r, v * r[:, None] * (f64(g) if g is not None else 1.0)


def _check_e4m3(codes, scale, y, what):
    T, H = y.shape
    nb = -(-H // 128)
    blocks = np.zeros((T, nb * 128))
    blocks[:, :H] = np.abs(y)
    want = np.maximum(blocks.reshape(T, nb, 128).max(2), LEAST) / 448.0
    assert_within(f64(scale), want, 66 * U * want, what + " scale")
    s = np.repeat(f64(scale), 128, 1)[:, :H]
    q, t = f64(codes), y / s
    # the quotient carries y's error and two roundings
    bound = 0.5 * e4m3_step(np.maximum(np.abs(q), np.abs(t))) + 80 * U * np.abs(t)
    assert_within(q, t, bound, what + " codes")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("T,H,pad,shift", [
    (1, 1, 0, 0), (3, 7, 0, 0), (2, 127, 1, 0), (5, 128, 0, 0), (4, 129, 7, 8), (1, 8192, 0, 0),
    (7, 8192, 8, 0), (33, 4099, 5, 0), (3, 4099, 0, 1), (2, 4104, 0, 3), (3, 16384, 0, 0),
    (2, 40000, 0, 0), (2, 33001, 0, 0), (700, 40, 0, 0), (403, 512, 8, 0), (350, 1001, 0, 0),
    (306, 1500, 0, 0), (310, 8200, 0, 0), (305, 5001, 0, 1), (1100, 40, 0, 0), (2000, 500, 12, 0),
    (1030, 511, 0, 0), (200, 8192, 0, 0), (400, 4099, 0, 0)])
def test_norm(dtype, eight, T, H, pad, shift):
    need_gpu()
    x, res, g = _inputs(T, H, dtype, 10 * H + T)
    dx, _ = placed(x, pad, shift)
    dr, _ = placed(res, pad, shift)
    dg, _ = placed(g[None], 0, shift)
    empty = torch.full((T, H), float("nan")).to(TORCH[dtype])
    ds, sbuf = placed(empty, pad, shift)
    out = "e4m3" if eight else dtype
    dy, ybuf = placed(torch.full((T, H), float("nan")).to(TORCH[out]), pad, shift)
    scale = torch.full((T, -(-H // 128)), float("nan"), device="cuda") if eight else None
    rstd = torch.full((T,), float("nan"), device="cuda")
    ar.ar_rmsnorm(dx, dr, dg, EPS, ds, dy, scale, rstd, T, H, dtype, out, ldx=H + pad,
                  ldres=H + pad, ldsum=H + pad, ldy=H + pad)
    torch.cuda.synchronize()
    want = (x.float() + res.float()).to(TORCH[dtype])
    assert torch.equal(ds.cpu(), want)                       # one add, one rounding
    v, r, y = _forward64(x, res, g)
    assert_within(f64(rstd), r, 48 * U * r, "rstd")
    if eight:
        _check_e4m3(dy, scale, y, "norm")
    else:
        assert_within(f64(dy), y, 64 * U * np.abs(y) + half(y, dtype), "y")
    assert untouched(sbuf, T, H, pad, shift) and untouched(ybuf, T, H, pad, shift)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_norm_without_residual_weight_and_sum(dtype):
    need_gpu()
    T, H = 5, 1000
    x, _, _ = _inputs(T, H, dtype, 3)
    y = torch.empty(T, H, dtype=TORCH[dtype], device="cuda")
    ar.ar_rmsnorm(x.cuda(), None, None, EPS, None, y, None, None, T, H, dtype)
    _, _, want = _forward64(x, None, None)
    assert_within(f64(y), want, 64 * U * np.abs(want) + half(want, dtype), "y")


@pytest.mark.parametrize("H", [1024, 33001])
def test_norm_in_place(H):
    """sum over the residual and y over x give what separate buffers give."""
    need_gpu()
    T = 6
    x, res, g = (t.cuda() for t in _inputs(T, H, "bf16", 4))
    s, y = torch.empty_like(x), torch.empty_like(x)
    ar.ar_rmsnorm(x, res, g, EPS, s, y, None, None, T, H, "bf16")
    ar.ar_rmsnorm(x, res, g, EPS, res, x, None, None, T, H, "bf16")
    assert torch.equal(s, res) and torch.equal(y, x)


def test_norm_zero_rows_and_zero_values():
    need_gpu()
    H = 300
    y = torch.full((1, H), 7.0, device="cuda")
    ar.ar_rmsnorm(None, None, None, EPS, None, y, None, None, 0, H, "fp32")
    torch.cuda.synchronize()
    assert bool((y == 7.0).all())
    x = torch.zeros(2, H, device="cuda")
    q = torch.ones(2, H, device="cuda").to(torch.float8_e4m3fn)
    scale = torch.empty(2, 3, device="cuda")
    ar.ar_rmsnorm(x, None, None, EPS, None, q, scale, None, 2, H, "fp32", "e4m3")
    assert bool((q.float() == 0).all())
    assert bool((scale == float(np.float32(LEAST) / np.float32(448.0))).all())


def test_norm_nan_stays_in_its_place():
    """A NaN weight: its element is the NaN code, its block keeps a finite scale."""
    need_gpu()
    T, H = 2, 512
    x, res, g = _inputs(T, H, "bf16", 5)
    g[200] = float("nan")
    q = torch.empty(T, H, device="cuda").to(torch.float8_e4m3fn)
    scale = torch.empty(T, 4, device="cuda")
    ar.ar_rmsnorm(x.cuda(), res.cuda(), g.cuda(), EPS, None, q, scale, None, T, H, "bf16", "e4m3")
    nan = torch.isnan(q.float()).cpu()
    assert bool(nan[:, 200].all()) and int(nan.sum()) == T
    g[200] = 0.0
    _check_e4m3(torch.where(nan, 0.0, q.float().cpu()), scale, _forward64(x, res, g)[2], "nan")


def test_norm_row_with_nan_or_infinity():
    """The row of a NaN is NaN; beside an infinity everything finite is 0 and
    the infinity itself NaN; other rows are as they would be."""
    need_gpu()
    x, res, g = _inputs(3, 256, "fp32", 6)
    clean = torch.empty(3, 256, device="cuda")
    ar.ar_rmsnorm(x.cuda(), res.cuda(), g.cuda(), EPS, None, clean, None, None, 3, 256, "fp32")
    x[0, 5], x[2, 9] = float("nan"), float("inf")
    y = torch.empty(3, 256, device="cuda")
    ar.ar_rmsnorm(x.cuda(), res.cuda(), g.cuda(), EPS, None, y, None, None, 3, 256, "fp32")
    assert bool(torch.isnan(y[0]).all()) and torch.equal(y[1], clean[1])
    assert bool(torch.isnan(y[2, 9])) and int((y[2] == 0).sum()) == 255


def _grad64(dy, dsum, s, g, r):
    n = f64(s) * r[:, None]
    gd = f64(dy) * (f64(g) if g is not None else 1.0)
    inner = (gd * n).mean(1, keepdims=True)
    extra = f64(dsum) if dsum is not None else np.zeros_like(n)
    dx = r[:, None] * (gd - n * inner) + extra
    # every product and sum of the formula, in magnitudes
    size = r[:, None] * (np.abs(gd) + np.abs(n) * np.abs(gd * n).mean(1, keepdims=True))
    return dx, 96 * U * (size + np.abs(extra)), (f64(dy) * n).sum(0), np.abs(f64(dy) * n).sum(0)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,H,pad,shift", [
    (1, 1, 0, 0), (1, 8192, 0, 0), (3, 7, 2, 0), (305, 264, 0, 0), (700, 129, 0, 1),
    (40, 4099, 5, 0), (5, 16384, 0, 0), (3, 20000, 0, 0), (3, 20001, 0, 0), (1300, 40, 0, 0),
    (2500, 512, 0, 0), (900, 1001, 0, 0), (650, 4096, 8, 0), (611, 2049, 0, 0), (330, 9000, 0, 0)])
def test_norm_grad(dtype, T, H, pad, shift):
    need_gpu()
    s, dsum, g = _inputs(T, H, dtype, 20 * H + T)
    dy = randn(T + H, T, H).to(TORCH[dtype])
    r = (1.0 / np.sqrt((f64(s) ** 2).mean(1) + EPS)).astype(np.float32)
    through = T % 2 == 1
    bufs = [placed(t, pad, shift)[0] for t in (dy, dsum, s)]
    dx, xbuf = placed(torch.full((T, H), float("nan")).to(TORCH[dtype]), pad, shift)
    dgamma = torch.full((H,), float("nan"), device="cuda")
    work = torch.full((min(T, 512) * H,), float("nan"), device="cuda")
    ar.ar_rmsnorm_grad(bufs[0], bufs[1] if through else None, bufs[2], g.cuda(),
                       torch.from_numpy(r).cuda(), dx, dgamma, work, work.numel() * 4, T, H,
                       dtype, lddy=H + pad, lddtotal=H + pad if through else 0,
                       ldtotal=H + pad, lddx=H + pad)
    want, bound, dg, size = _grad64(dy, dsum if through else None, s, g, r.astype(np.float64))
    assert_within(f64(dx), want, bound + half(want, dtype), "dx")
    # a column's sum: at most T / 256 + 1 adds in a CTA, 17 partial rows, a tree
    assert_within(f64(dgamma), dg, (T / 256 + 32) * U * size + 1e-40, "dgamma")
    assert untouched(xbuf, T, H, pad, shift)


def test_norm_grad_against_differences():
    """Central differences of the binary64 forward (h = 1e-4: truncation below
    1e-6 of the slope's scale) against the kernel's binary32 gradient."""
    need_gpu()
    T, H, h = 3, 40, 1e-4
    x, res, g = _inputs(T, H, "fp32", 8)
    dy = randn(9, T, H).float()
    v = (x.float() + res.float())
    _, r, _ = _forward64(v, None, g)
    dx = torch.empty(T, H, device="cuda")
    dgamma = torch.empty(H, device="cuda")
    work = torch.empty(T * H, device="cuda")
    ar.ar_rmsnorm_grad(dy.cuda(), None, v.cuda(), g.cuda(),
                       torch.from_numpy(r.astype(np.float32)).cuda(), dx, dgamma, work,
                       4 * T * H, T, H, "fp32")

    def loss(v64, g64):
        rr = 1.0 / np.sqrt((v64 * v64).mean(1) + EPS)
        return (v64 * rr[:, None] * g64 * f64(dy)).sum()
    v64, g64 = f64(v), f64(g)
    for t, i in [(0, 0), (1, 17), (2, 39)]:
        step = np.zeros_like(v64)
        step[t, i] = h
        slope = (loss(v64 + step, g64) - loss(v64 - step, g64)) / (2 * h)
        assert abs(float(dx[t, i]) - slope) <= 1e-5
    for i in (0, 21, 39):
        step = np.zeros_like(g64)
        step[i] = h
        slope = (loss(v64, g64 + step) - loss(v64, g64 - step)) / (2 * h)
        assert abs(float(dgamma[i]) - slope) <= 1e-5


def test_norm_grad_parts_and_zero_rows():
    need_gpu()
    T, H = 9, 520
    s, _, g = _inputs(T, H, "bf16", 11)
    dy = randn(12, T, H).bfloat16().cuda()
    r = torch.rsqrt(s.float().square().mean(1) + EPS).cuda()
    s, g = s.cuda(), g.cuda()
    dx, dx2 = torch.empty_like(s), torch.empty_like(s)
    dgamma, work = torch.empty(H, device="cuda"), torch.empty(T * H, device="cuda")
    ar.ar_rmsnorm_grad(dy, None, s, g, r, dx, dgamma, work, 4 * T * H, T, H, "bf16")
    ar.ar_rmsnorm_grad(dy, None, s, g, r, dx2, None, None, 0, T, H, "bf16")
    assert torch.equal(dx, dx2)
    ar.ar_rmsnorm_grad(dy, None, s, g, r, dy, None, None, 0, T, H, "bf16")    # over dy
    assert torch.equal(dx, dy)
    dgamma.fill_(3.0)
    ar.ar_rmsnorm_grad(None, None, None, None, None, None, dgamma, None, 0, 0, H, "bf16")
    assert bool((dgamma == 0).all())


def test_norm_in_a_graph_on_another_stream():
    need_gpu()
    T, H = 16, 2048
    x, res, g = (t.cuda() for t in _inputs(T, H, "bf16", 13))
    s, y = torch.empty_like(x), torch.empty_like(x)
    want_s, want_y = torch.empty_like(x), torch.empty_like(x)
    ar.ar_rmsnorm(x, res, g, EPS, want_s, want_y, None, None, T, H, "bf16")
    torch.cuda.synchronize()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        ar.ar_rmsnorm(x, res, g, EPS, s, y, None, None, T, H, "bf16", stream=stream)
    for _ in range(2):
        s.zero_(), y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(s, want_s) and torch.equal(y, want_y)
