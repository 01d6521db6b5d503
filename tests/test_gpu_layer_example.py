"""The layer operators together, as examples/moe_layer.py uses them.

Bounds (2-norm, relative).  serve(): the plain form skips the E4M3 rounding of the
activations between the two products (at most 2^-4 of an element, about 2^-5.3 on
average over a binade, so below 0.04) and the bf16 roundings (2^-9 each, four of
them).  train(): bf16 roundings of the normed rows, of the experts' results and of
two gradients, 2^-9 each, in chains of at most five: 0.01."""
import os
import sys

import pytest
import torch

from gpu_helpers import need_gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,hidden,inner,experts,top,ranks", [
    (1, 512, 128, 8, 2, 4), (64, 1024, 384, 16, 4, 8), (300, 640, 256, 5, 3, 2)])
def test_layer(tokens, hidden, inner, experts, top, ranks):
    need_gpu()
    import moe_layer
    layer = moe_layer.Layer(tokens, hidden, inner, experts, top, ranks, seed=tokens)
    out = layer.serve()
    assert moe_layer.off(out, layer.serve_plain()) < 0.05
    for name, (got, want) in layer.train().items():
        assert moe_layer.off(got, want) < 0.01, name
    layer.close()
    torch.cuda.synchronize()
