"""ar_rmsnorm and its gradient where the other norm tests do not reach: the E4M3
arithmetic bit for bit, rows of very small and very large values, and every form
that the number of rows, their width and their alignment choose.

Bounds.  y and dx: the 64 u and 96 u of the terms' magnitudes that test_gpu_norm.py
derives; they are relative, so they hold at every scale of s.  dgamma: a thread adds
one product a row of its CTA, of which there are 152 at least where rows repeat
(ceil(T / 152) adds); at most 16 groups of a CTA are then joined (15), at most 512
partial rows by 32 threads (16) and a tree (5); the product carries two roundings.
Together below (ceil(T / 152) + 38) u of the column's magnitudes."""
import numpy as np
import pytest
import torch

import all_reduce_reduction_gb300 as ar
from gpu_helpers import need_gpu
from layer_helpers import (LEAST, TORCH, U, assert_within, e4m3_step, f64, half, placed, randn,
                           untouched)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,H", [(3, 512), (2, 1000), (1100, 300), (700, 2048)])
def test_scale_and_codes_are_products_with_rounded_reciprocals(dtype, T, H):
    """Rows of +-1 with eps = 0 have r = 1 exactly, so that y is the weight with
    the row's signs, and every later operation is one binary32 rounding."""
    need_gpu()
    x = torch.where(randn(H, T, H) < 0, -1.0, 1.0).to(TORCH[dtype])
    g = (randn(H + 1, H) * torch.exp2(torch.randint(-40, 40, (H,), generator=torch.Generator()
                                                    .manual_seed(H)).double()))
    g = g.to(TORCH[dtype])
    nb = -(-H // 128)
    q = torch.empty(T, H, device="cuda").to(torch.float8_e4m3fn)
    scale = torch.empty(T, nb, device="cuda")
    ar.ar_rmsnorm(x.cuda(), None, g.cuda(), 0.0, None, q, scale, None, T, H, dtype, "e4m3")
    y = (x.float() * g.float()).numpy()
    top = np.zeros((T, nb * 128), np.float32)
    top[:, :H] = np.abs(y)
    top = np.maximum(top.reshape(T, nb, 128).max(2), np.float32(LEAST))
    want = top * (np.float32(1.0) / np.float32(448.0))
    assert np.array_equal(scale.cpu().numpy(), want)
    inverse = np.repeat(np.float32(1.0) / want, 128, 1)[:, :H]
    codes = torch.from_numpy(y * inverse).to(torch.float8_e4m3fn)
    assert torch.equal(q.cpu().view(torch.uint8), codes.view(torch.uint8))


def _grad64(dy, dsum, s, g, r):
    """(dx, its bound before the output's rounding, dgamma, dgamma's magnitudes)."""
    n, r = f64(s) * r.astype(np.float64)[:, None], r.astype(np.float64)[:, None]
    gd = f64(dy) * f64(g)
    extra = f64(dsum) if dsum is not None else np.zeros_like(n)
    dx = r * (gd - n * (gd * n).mean(1, keepdims=True)) + extra
    size = r * (np.abs(gd) + np.abs(n) * np.abs(gd * n).mean(1, keepdims=True)) + np.abs(extra)
    return dx, 96 * U * size, (f64(dy) * n).sum(0), np.abs(f64(dy) * n).sum(0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("scale", [1e-20, 1e17])
@pytest.mark.parametrize("T,H", [(5, 1000), (3, 20001), (2500, 512), (400, 8192)])
def test_gradient_of_very_small_and_very_large_rows(dtype, scale, T, H):
    """r^3 leaves binary32 where neither r nor dx does."""
    need_gpu()
    s = (randn(T, T, H) * scale).to(TORCH[dtype])
    dy, g = randn(H, T, H).to(TORCH[dtype]), (1 + 0.2 * randn(7, H)).to(TORCH[dtype])
    r = (1.0 / np.sqrt((f64(s) ** 2).mean(1))).astype(np.float32)
    dx = torch.empty(T, H, dtype=TORCH[dtype], device="cuda")
    ar.ar_rmsnorm_grad(dy.cuda(), None, s.cuda(), g.cuda(), torch.from_numpy(r).cuda(), dx, None,
                       None, 0, T, H, dtype)
    want, bound, _, _ = _grad64(dy, None, s, g, r)
    assert_within(f64(dx), want, bound + half(want, dtype), "dx")


# rows, width, elements after each row, elements before the first
ONE_WARP = [(1100, 40, 0, 0), (1100, 200, 3, 0), (1030, 255, 0, 1), (1500, 130, 8, 0)]
FOUR_UNITS = [(700, 1001, 0, 1), (200, 4001, 0, 0), (450, 1500, 1, 0), (300, 4096, 0, 0),
              (700, 1024, 8, 0)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("T,H,pad,shift", ONE_WARP + FOUR_UNITS)
def test_norm_of_many_rows(dtype, eight, T, H, pad, shift):
    """A warp a row, and four units a thread, on and off the vector path."""
    need_gpu()
    eps = 1e-5
    x, res = randn(T, T, H).to(TORCH[dtype]), (randn(H, T, H) * 8).to(TORCH[dtype])
    g = (1 + 0.2 * randn(T + H, H)).to(TORCH[dtype])
    out = "e4m3" if eight else dtype
    nan = torch.full((T, H), float("nan"))
    dx, dr, dg = placed(x, pad, shift)[0], placed(res, pad, shift)[0], placed(g[None], 0, shift)[0]
    ds, sbuf = placed(nan.to(TORCH[dtype]), pad, shift)
    dy, ybuf = placed(nan.to(TORCH[out]), pad, shift)
    scale = torch.full((T, -(-H // 128)), float("nan"), device="cuda") if eight else None
    rstd = torch.full((T,), float("nan"), device="cuda")
    ld = H + pad
    ar.ar_rmsnorm(dx, dr, dg, eps, ds, dy, scale, rstd, T, H, dtype, out, ldx=ld, ldres=ld,
                  ldsum=ld, ldy=ld)
    v = f64(x) + f64(res)
    r = 1.0 / np.sqrt((v * v).mean(1) + eps)
    y = v * r[:, None] * f64(g)
    assert torch.equal(ds.cpu(), (x.float() + res.float()).to(TORCH[dtype]))
    assert_within(f64(rstd), r, 48 * U * r, "rstd")
    assert untouched(sbuf, T, H, pad, shift) and untouched(ybuf, T, H, pad, shift)
    if not eight:
        assert_within(f64(dy), y, 64 * U * np.abs(y) + half(y, dtype), "y")
        return
    nb = -(-H // 128)
    top = np.zeros((T, nb * 128))
    top[:, :H] = np.abs(y)
    top = np.maximum(top.reshape(T, nb, 128).max(2), LEAST) / 448.0
    assert_within(f64(scale), top, 66 * U * top, "scale")      # y's 64 u and two products
    q, t = f64(dy), y / np.repeat(f64(scale), 128, 1)[:, :H]
    assert_within(q, t, 0.5 * e4m3_step(np.maximum(np.abs(q), np.abs(t))) + 80 * U * np.abs(t),
                  "codes")


# the ring: groups of one row with warps left over, one row a CTA, ragged ends, several
# turns; without it: groups, one row, units past the registers; few rows
GRADIENT = [(1999, 2560, 0, 0), (2500, 512, 0, 0), (1000, 4096, 0, 0), (701, 4100, 4, 0),
            (650, 8192, 0, 0), (1999, 1288, 8, 0), (1999, 257, 0, 1), (1300, 1001, 0, 1),
            (700, 4001, 3, 0), (330, 9000, 0, 0), (330, 16500, 0, 0), (160, 20001, 0, 0),
            (40, 8192, 0, 0), (37, 4099, 0, 0)]


def _gradient(bufs, dsum, g, rstd, dx, T, H, ld, dtype):
    dgamma = torch.full((H,), float("nan"), device="cuda")
    work = torch.full((min(T, ar.AR_NORM_GRAD_ROWS) * H,), float("nan"), device="cuda")
    ar.ar_rmsnorm_grad(bufs[0], dsum, bufs[1], g, rstd, dx, dgamma, work, 4 * work.numel(), T, H,
                       dtype, lddy=ld, lddtotal=ld if dsum is not None else 0, ldtotal=ld, lddx=ld)
    return dgamma


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("through", [True, False])
@pytest.mark.parametrize("T,H,pad,shift", GRADIENT)
def test_gradient_with_and_without_the_sums_own(dtype, through, T, H, pad, shift):
    """dx and dgamma, and dx written over each of dsum, dy and s: the same bits."""
    need_gpu()
    s, dy = (4 * randn(T, T, H)).to(TORCH[dtype]), randn(H, T, H).to(TORCH[dtype])
    dsum = randn(T + H, T, H).to(TORCH[dtype]) if through else None
    g = (1 + 0.2 * randn(3, H)).to(TORCH[dtype])
    r = (1.0 / np.sqrt((f64(s) ** 2).mean(1) + 1e-5)).astype(np.float32)
    rstd, dg, ld = torch.from_numpy(r).cuda(), g.cuda(), H + pad

    def fresh():
        return [placed(t, pad, shift)[0] if t is not None else None for t in (dy, s, dsum)]
    bufs = fresh()
    dx, xbuf = placed(torch.full((T, H), float("nan")).to(TORCH[dtype]), pad, shift)
    dgamma = _gradient(bufs, bufs[2], dg, rstd, dx, T, H, ld, dtype)
    want, bound, wg, size = _grad64(dy, dsum, s, g, r)
    assert_within(f64(dx), want, bound + half(want, dtype), "dx")
    assert_within(f64(dgamma), wg, (-(-T // 152) + 38) * U * size + 1e-40, "dgamma")
    assert untouched(xbuf, T, H, pad, shift)
    for over in (2, 0, 1) if through else (0, 1):
        again = fresh()
        dgamma2 = _gradient(again, again[2], dg, rstd, again[over], T, H, ld, dtype)
        assert torch.equal(again[over], dx) and torch.equal(dgamma2, dgamma), over
