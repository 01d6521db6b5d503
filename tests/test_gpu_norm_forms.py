"""ar_rmsnorm and its gradient where the other norm tests do not reach: the E4M3
arithmetic bit for bit, rows of very small and very large values.

Bounds of the gradient.  dx: the 96 u of its terms' magnitudes that
test_gpu_norm.py derives; they are relative, so they hold at every scale of s."""
import numpy as np
import pytest
import torch

import all_reduce_reduction_gb300 as ar
from gpu_helpers import need_gpu
from layer_helpers import LEAST, TORCH, U, assert_within, f64, half, randn

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
