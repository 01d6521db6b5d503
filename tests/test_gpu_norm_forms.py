"""ar_rmsnorm and its gradient where the other norm tests do not reach: the E4M3
arithmetic bit for bit."""
import numpy as np
import pytest
import torch

import all_reduce_reduction_gb300 as ar
from gpu_helpers import need_gpu
from layer_helpers import LEAST, TORCH, randn

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
