"""ar_moe_return where every CTA takes several jobs: the rows and weights of a job are
read while the one before is at work.  Bit for bit, as in test_gpu_moe.py, whose fold and
order these cases share."""
import numpy as np
import pytest
import torch

import all_reduce_reduction_gb300 as ar
from gpu_helpers import need_gpu
from layer_helpers import TORCH, placed, randn, untouched
from test_gpu_moe import _fold32, _ids, _order

pytestmark = pytest.mark.gpu

# tokens, choices, experts, width, elements after each row, before the first.  A job is
# 256 units of a row (8 or 4 elements aligned, 4 otherwise); 456 CTAs take them in turn.
JOBS = [(700, 8, 16, 2056, 0, 0), (300, 9, 16, 8192, 0, 0), (5000, 3, 8, 264, 0, 0),
        (700, 8, 16, 2049, 0, 1), (3000, 5, 8, 517, 3, 1), (900, 17, 32, 1040, 0, 0),
        (4003, 1, 4, 1000, 0, 0), (250, 32, 64, 4100, 4, 0)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("T,K,E,H,pad,shift", JOBS)
def test_return_of_many_jobs(dtype, weighted, T, K, E, H, pad, shift):
    need_gpu()
    ids = _ids(T, K, E, H + T, 0, 2 * E)                     # half of the experts elsewhere
    ids[::7] = E                                             # tokens without any here
    _, row_of, _ = _order(ids, E)
    n = int(row_of.max()) + 1                                # the rows that are here
    y = randn(T + H, n, H).float().to(TORCH[dtype])
    w = np.random.default_rng(T).random((T, K)).astype(np.float32) if weighted else None
    rows, _ = placed(y, pad, shift)
    out, buf = placed(torch.full((T, H), float("nan")).to(TORCH[dtype]), pad, shift)
    ar.ar_moe_return(rows, n, torch.from_numpy(row_of).int().cuda(),
                     torch.from_numpy(w).cuda() if weighted else None, out, T, K, H, dtype,
                     ldrows=H + pad, ldout=H + pad)
    want = torch.from_numpy(_fold32(y.float().numpy(), row_of, w)).to(TORCH[dtype])
    assert torch.equal(out.cpu(), want)
    assert bool((out[::7] == 0).all())
    assert untouched(buf, T, H, pad, shift)
