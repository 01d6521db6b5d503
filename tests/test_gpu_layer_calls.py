"""The layer operators called as a program calls them: with tensors alone."""
import os
import sys

import numpy as np
import pytest
import torch

import all_reduce_reduction_gb300 as ar
from gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_route_of_a_topk(dtype):
    """Ids as torch.topk gives them (8 bytes), or narrowed, with no width said."""
    need_gpu()
    T, K, E = 300, 4, 32
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.topk(torch.randn(T, E, generator=g, device="cuda"), K, dim=1).indices.to(dtype)
    offsets = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    row_of, src = (torch.empty(T * K, dtype=torch.int32, device="cuda") for _ in range(2))
    ar.ar_moe_route(ids, T, K, E, offsets, row_of, src)
    flat = ids.cpu().numpy().reshape(-1)
    order = np.argsort(flat, kind="stable")
    assert np.array_equal(src.cpu().numpy(), order)
    assert np.array_equal(offsets.cpu().numpy(), np.searchsorted(flat[order], np.arange(E + 1)))
    assert np.array_equal(row_of.cpu().numpy()[order], np.arange(T * K))


def test_the_example_reads_what_its_products_report(monkeypatch):
    """Every product has the layer's status word, and a word that is set stops the step."""
    need_gpu()
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                    "examples"))
    import moe_layer
    layer = moe_layer.Layer(8, 256, 128, 4, 2, 2)
    product, seen = ar.ar_matmul8, []

    def recorded(*args, status=None, **kw):
        seen.append(status)
        product(*args, status=status, **kw)
    monkeypatch.setattr(ar, "ar_matmul8", recorded)
    layer.serve()
    layer.check()
    assert len(seen) == 2 and all(s is layer.status for s in seen)
    layer.status.fill_(ar.AR_ERR_TIMEOUT)
    with pytest.raises(ar.ArError) as e:
        layer.check()
    assert e.value.code == ar.AR_ERR_TIMEOUT
    layer.close()
