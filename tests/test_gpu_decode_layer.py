"""The calls of a decode step together, as examples/decode_layer.py uses them: prompts
into the caches, then steps of one captured graph while the sequences grow.

Bounds (2-norm, relative).  Attention's sum: the plain form starts from the same cache and
the same q; the outputs are rounded to bf16 (2^-9), the projections of R ranks again, and
their sum once more: three roundings of 2^-9, below 0.006 (a rounding is off by half a
step at most, 2^-9 of the value; those of the ranks add up like their squares).  The layer's
output: the ranks' results and their sum, two roundings, and h with 11 bits of its
largest neighbour's: below 0.006 as well.  E4M3 rows: half a step, 2^-4 of an element, and
2^-10 of the row's largest below 2^-6 of the scale's range."""
import os
import sys

import pytest
import torch

from gpu_helpers import need_gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["e4m3", "bf16"])
@pytest.mark.parametrize("sequences,hidden,heads,kv,dim,page,inner,experts,top,ranks,lengths", [
    (1, 512, 8, 2, 64, 16, 128, 8, 2, 2, [40]),
    (5, 1024, 16, 4, 128, 16, 256, 8, 3, 4, [1, 130, 15, 64, 300]),
    (16, 640, 10, 5, 80, 8, 160, 10, 4, 5, [7 * b + 1 for b in range(16)])])
def test_decode(cache, sequences, hidden, heads, kv, dim, page, inner, experts, top, ranks,
                lengths):
    need_gpu()
    import all_reduce_reduction_gb300 as ar
    import decode_layer
    d = decode_layer.Decoder(sequences, max(lengths) + 40, hidden, heads, kv, dim, page, inner,
                             experts, top, ranks, cache, seed=hidden)
    g = torch.Generator(device="cuda").manual_seed(2)
    d.prompt(torch.randn(sum(lengths), hidden, generator=g, device="cuda").bfloat16(), lengths)
    # what was written comes back
    for c, (k, v, offsets) in zip(d.caches, d.prompt_rows):
        back = [torch.zeros(sum(lengths), d.kv * dim, dtype=torch.bfloat16, device="cuda")
                for _ in "kv"]
        ar.ar_cache_read(*d._cache_args(c), offsets, *back, sum(lengths), sequences, d.kv, dim,
                         "bf16", cache)
        for got, want in zip(back, (k, v)):
            if cache == "bf16":
                assert torch.equal(got, want)
                continue
            got, want = (t.float().view(-1, d.kv, dim) for t in (got, want))
            top_of = want.abs().amax(2, keepdim=True)
            bound = want.abs() * (2.0 ** -4 + 2.0 ** -8) + top_of * 2.0 ** -16
            assert bool(((got - want).abs() <= bound).all())
    graph = d.captured()
    for _ in range(20):                                       # across the ends of pages
        d.x.copy_(torch.randn(sequences, hidden, generator=g, device="cuda"))
        graph.replay()
    for _ in range(3):
        d.x.copy_(torch.randn(sequences, hidden, generator=g, device="cuda"))
        graph.replay()
        d.check()
        attention, out = d.plain()
        assert decode_layer.off(d.summed[0], attention) < 0.006
        assert decode_layer.off(d.out[0], out) < 0.006
        assert torch.equal(d.out[0], d.out[-1])
    assert d.lens.tolist() == [n + 23 for n in lengths]
    d.close()
    torch.cuda.synchronize()
