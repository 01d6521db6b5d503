"""Calls of a decode step's operators that their documentation allows: several at once, captured
and replayed beside eager ones, the most heads, the widest rows."""
import numpy as np
import pytest
import torch

import all_reduce_reduction_gb300 as ar
from cache_helpers import Cache, quantised
from gpu_helpers import need_gpu
from layer_helpers import TORCH, randn
from test_gpu_cache_attention import _check as _check_attention
from test_gpu_moe_layer import Layer, _ids

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_experts_at_once_with_a_workspace_each(dtype):
    """Two streams and a graph on a third, over and over: the same bits as one after another."""
    need_gpu()
    T, K, E, H, F = 12, 3, 8, 1024, 384
    layer = Layer(E, H, F)
    sets = []
    for i in range(3):
        x = randn(i, T, H).to(TORCH[dtype]).cuda()
        sets.append(dict(x=x, ids=_ids(T, K, E, i), w=torch.rand(T, K, device="cuda"),
                         out=torch.empty_like(x), work=torch.empty(T * K * (F + 128), device="cuda"),
                         stream=torch.cuda.Stream()))

    def call(x, ids, w, out, work, stream):
        ar.ar_moe_layer(x, ids, w, layer.up, layer.us, layer.down, layer.ds, out, work,
                        4 * work.numel(), T, K, E, H, F, dtype, stream=stream)
    want = []
    for s in sets:
        call(**{**s, "stream": None})
        torch.cuda.synchronize()
        want.append(s["out"].clone())
        s["out"].fill_(7)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=sets[2]["stream"]):
        call(**sets[2])
    for _ in range(20):
        call(**sets[0])
        with torch.cuda.stream(sets[2]["stream"]):
            graph.replay()
        call(**sets[1])
    torch.cuda.synchronize()
    for s, w in zip(sets, want):
        assert torch.equal(s["out"], w)


def test_a_workspace_serves_calls_of_any_size_in_turn():
    need_gpu()
    work = torch.full((64 * 8 * (512 + 128),), float("nan"), device="cuda")
    layers = [Layer(4, 256, 512, 1), Layer(3, 100, 33, 2)]
    for dtype in ("fp16", "fp32", "bf16"):
        for layer, T, K in ((layers[0], 64, 4), (layers[1], 1, 1), (layers[0], 2, 2),
                            (layers[1], 20, 3)):
            x = randn(T, T, layer.H).to(TORCH[dtype]).cuda()
            ids, outs = _ids(T, K, layer.E, T), [torch.empty_like(x) for _ in range(2)]
            for out, buf in zip(outs, (work, torch.zeros_like(work))):
                ar.ar_moe_layer(x, ids, None, layer.up, layer.us, layer.down, layer.ds, out, buf,
                                4 * buf.numel(), T, K, layer.E, layer.H, layer.F, dtype,
                                ldup=layer.ld[0], lddown=layer.ld[1])
            torch.cuda.synchronize()
            assert torch.equal(*outs) and bool(torch.isfinite(outs[0]).all())


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp16", "e4m3"), ("fp32", "fp32")])
@pytest.mark.parametrize("heads,kv,D", [(1024, 1, 16), (1024, 1024, 8), (1024, 32, 64),
                                        (1000, 8, 24)])
def test_attention_of_the_most_heads(dtype, cache, heads, kv, D):
    _check_attention([5, 70], heads, kv, D, 16, dtype, cache, seed=D)


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp16", "e4m3"), ("fp32", "e4m3")])
@pytest.mark.parametrize("heads,D", [(1024, 256), (1024, 255), (1000, 1), (1, 256), (3, 250)])
def test_rows_of_the_most_heads_into_the_cache_and_back(dtype, cache, heads, D):
    need_gpu()
    lens, new, page = [5, 2, 0, 3], [3, 2, 0, 1], 2
    c = Cache(lens, heads, D, page, dtype, cache)
    T = sum(new)
    offsets = torch.tensor([0] + new).cumsum(0).int().cuda()
    rows = [randn(i, T, heads * D).to(TORCH[dtype]).cuda() for i in range(2)]
    ar.ar_cache_write(*rows, *c.args(), offsets, T, 4, heads, D, dtype, cache, **c.strides())
    back = [torch.full_like(r, 7) for r in rows]
    ar.ar_cache_read(*c.args(), offsets, *back, T, 4, heads, D, dtype, cache, **c.strides())
    torch.cuda.synchronize()
    for r, b in zip(rows, back):
        want = r
        if c.eight:
            codes, scale = quantised(r.view(T, heads, D))
            value = codes.view(torch.float8_e4m3fn).float().numpy() * scale.numpy()[..., None]
            want = torch.from_numpy(value.astype(np.float32)).to(TORCH[dtype]).view(T, -1).cuda()
        assert torch.equal(b, want)
