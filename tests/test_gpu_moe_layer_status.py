"""ar_moe_layer's status word: the last word of its workspace."""
import pytest
import torch

import all_reduce_reduction_gb300 as ar
from gpu_helpers import need_gpu
from layer_helpers import TORCH
from test_gpu_moe_layer import Layer, _ids

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,K,E,H,F", [
    (1, 1, 1, 16, 1), (1, 1, 1, 16, 97), (1, 1, 1, 16, 129), (1, 1, 1, 16, 2049), (3, 2, 4, 40, 33),
    (1, 1, 1, 16, 6145), (2, 8, 16, 64, 800), (64, 8, 8, 16, 65)])
def test_ok_after_a_call_and_nothing_past_it(dtype, T, K, E, H, F):
    """Whatever the workspace held; sizes whose rows of h leave the least room beside it."""
    need_gpu()
    layer = Layer(E, H, F)
    x = torch.randn(T, H, device="cuda").to(TORCH[dtype])
    ids, out = _ids(T, K, E, 1), torch.empty_like(x)
    n = T * K * (F + 128)
    first = None
    for fill in (0x7FC00000, 0, -1):
        work = torch.full((n + 8,), fill, dtype=torch.int32, device="cuda")
        ar.ar_moe_layer(x, ids, None, layer.up, layer.us, layer.down, layer.ds, out, work, 4 * n,
                        T, K, E, H, F, dtype, ldup=layer.ld[0], lddown=layer.ld[1])
        torch.cuda.synchronize()
        assert int(work[n - 1]) == ar.AR_OK
        assert bool((work[n:] == fill).all())
        assert first is None or torch.equal(out, first)
        assert bool(torch.isfinite(out).all())
        first = out.clone()
