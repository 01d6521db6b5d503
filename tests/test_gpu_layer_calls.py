"""The layer operators called as a program calls them: with tensors alone."""
import os
import sys
import threading

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


def _every_call(T=64, K=2, E=4, H=256):
    """(calls without a stream, the tensors that they write)."""
    g = torch.Generator(device="cuda").manual_seed(2)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    n, kb = T * K, H // 128
    x, res, gamma = normal(T, H), normal(T, H), normal(H)
    ids = torch.topk(normal(T, E), K, dim=1).indices
    w, weights = torch.rand(T, K, generator=g, device="cuda"), normal(E * H, H).mul_(50)
    weights = weights.to(torch.float8_e4m3fn)
    sb = torch.rand(E, kb, kb, generator=g, device="cuda")
    out = {k: torch.zeros(*s, device="cuda") for k, s in dict(
        total=(T, H), scale=(T, kb), rstd=(T,), dx=(T, H), dgamma=(H,), work=(T * H,),
        rscale=(n, kb), y=(n, H), out=(T, H), drows=(n, H), dw=(T, K)).items()}
    out |= {k: torch.zeros(*s, dtype=torch.int32, device="cuda") for k, s in dict(
        offsets=(E + 1,), row_of=(T, K), src=(n,), status=(1,)).items()}
    out |= {k: torch.zeros(s, H, device="cuda").to(torch.float8_e4m3fn) for k, s in
            (("codes", T), ("rows", n))}
    o = out

    def calls():
        ar.ar_rmsnorm(x, res, gamma, 1e-6, o["total"], o["codes"], o["scale"], o["rstd"], T, H,
                      "fp32", "e4m3")
        ar.ar_moe_route(ids, T, K, E, o["offsets"], o["row_of"], o["src"])
        ar.ar_moe_dispatch(o["codes"], o["scale"], o["row_of"], o["rows"], o["rscale"], n, T, K, H,
                           "e4m3")
        ar.ar_matmul8(o["rows"], o["rscale"], weights, sb, o["offsets"], E, o["y"], n, H, H,
                      "fp32", status=o["status"])
        ar.ar_moe_return(o["y"], n, o["row_of"], w, o["out"], T, K, H, "fp32")
        ar.ar_moe_return_grad(o["out"], o["y"], n, o["row_of"], w, o["drows"], o["dw"], T, K, H,
                              "fp32")
        ar.ar_rmsnorm_grad(o["out"], None, o["total"], gamma, o["rstd"], o["dx"], o["dgamma"],
                           o["work"], 4 * T * H, T, H, "fp32")
    return calls, out


def _bits(out):
    return {k: t.view(torch.uint8).clone() for k, t in out.items() if k != "work"}


def test_calls_without_a_stream_take_the_current_one():
    """Captured on a side stream (anything launched elsewhere would end the capture), and
    from a thread with a stream of its own."""
    need_gpu()
    calls, out = _every_call()
    calls()
    torch.cuda.synchronize()
    want = _bits(out)
    assert int(out["status"]) == 0 and float(out["dw"].abs().sum()) > 0

    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        assert ar._current_stream() == side.cuda_stream
    with torch.cuda.graph(graph, stream=side):
        calls()
    for t in out.values():
        t.view(torch.uint8).zero_()
    torch.cuda.synchronize()
    assert float(out["dw"].abs().sum()) == 0                 # captured, not run
    graph.replay()
    torch.cuda.synchronize()
    got = _bits(out)
    assert all(torch.equal(got[k], want[k]) for k in want)

    seen = []

    def other():
        own = torch.cuda.Stream()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=own, capture_error_mode="thread_local"):
            calls()
        seen.append((ar._current_stream() == torch.cuda.current_stream().cuda_stream, g))
    thread = threading.Thread(target=other)
    thread.start()
    thread.join()
    assert seen and seen[0][0]
    for t in out.values():
        t.view(torch.uint8).zero_()
    seen[0][1].replay()
    torch.cuda.synchronize()
    got = _bits(out)
    assert all(torch.equal(got[k], want[k]) for k in want)
