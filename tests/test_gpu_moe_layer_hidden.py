"""What ar_moe_layer keeps of h between its launches, against the definition in binary64.

Bound: that of test_gpu_moe_layer.py, but for what h loses between the launches.  Where the
output has two bytes, h is two binary16 numbers of 11 bits that 16 neighbours scaled by a power
of two, the lowest bit of the second given away: off by one unit of the second, 2^-10 of it, and
the second is at most 2^-11 of h: r = 2^-21.  A tile's largest magnitude is at least 2^-1 after
scaling and a unit at least 2^-24: 2^-23 of the tile's largest more.  Where tiles of a block of
128 are brought to one scale, and in binary32, two numbers of 11 bits (2^-21) with the block's
largest at 2^14 or more: 2^-39 of it."""
import pytest
import torch

from gpu_helpers import need_gpu
from layer_helpers import TORCH, U, assert_within, half
from test_gpu_moe_layer import Layer, _ids

pytestmark = pytest.mark.gpu


def _blocks_largest(h, size):
    """The largest magnitude of the `size` neighbours of each element."""
    F = h.shape[1]
    padded = torch.nn.functional.pad(h.abs(), (0, -F % size)).unflatten(1, (-1, size))
    return padded.amax(2).repeat_interleave(size, 1)[:, :F]


def _exact(layer, x, ids, w, dtype):
    T = x.shape[0]
    H, F, K = layer.H, layer.F, ids.shape[1]
    hb, fb = -(-H // 128), -(-F // 128)
    i = {n: torch.arange(n, device="cuda") // 128 for n in (H, F, 2 * F)}
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    err, size = torch.zeros_like(out), torch.zeros_like(out)
    a1, a2 = (80 + 2 * hb) * U + (2.0 ** -21 if dtype == "fp32" else 0), (80 + 2 * fb) * U
    for e in sorted(set(ids.flatten().tolist())):
        t, k = torch.nonzero(ids == e, as_tuple=True)
        w1 = layer.up[e].float().double() * layer.us[e].double()[i[2 * F]][:, i[H]]
        w2 = layer.down[e].float().double() * layer.ds[e].double()[i[H]][:, i[F]]
        v = x[t].double()
        both = v @ w1.t()
        off = a1 * (v.abs() @ w1.abs().t()) + 2.0 ** -39 * (_blocks_largest(v, 128) @ w1.abs().t())
        (g, u), (dg, du) = both.split(F, 1), off.split(F, 1)
        act = g * torch.sigmoid(g)
        h = act * u
        dh = 1.1 * (u.abs() + du) * dg + act.abs() * du + 16 * U * h.abs()
        dh += 2.0 ** -21 * h.abs() + 2.0 ** -39 * _blocks_largest(h, 128)
        if dtype != "fp32":
            dh += 2.0 ** -23 * _blocks_largest(h, 16)
        each = h.abs() @ w2.abs().t()
        gate = w[t, k, None].double()
        out.index_add_(0, t, gate * (h @ w2.t()))
        err.index_add_(0, t, gate.abs() * (dh @ w2.abs().t() + a2 * each))
        size.index_add_(0, t, gate.abs() * each)
    return out, err + (K + 10) * U * size


def _check(layer, T, K, dtype, seed=0, ids=None, spoil=None):
    need_gpu()
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, layer.H, generator=g, device="cuda")
    if spoil is not None:
        spoil(x)
    x = x.to(TORCH[dtype])
    ids = _ids(T, K, layer.E, seed + 1) if ids is None else ids
    w = 0.5 + torch.rand(T, K, generator=g, device="cuda")
    out = torch.full((T, layer.H), float("nan"), device="cuda").to(TORCH[dtype])
    layer.call(x, ids, w, dtype, out)
    torch.cuda.synchronize()
    want, err = (a.cpu().numpy() for a in _exact(layer, x.float(), ids, w, dtype))
    assert_within(out.double().cpu().numpy(), want, err + half(want, dtype) * (1 + 1e-6), "out")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("H,F", [(16, 1), (64, 1), (64, 5), (32, 16), (48, 17), (64, 33), (16, 48),
                                 (64, 127), (16, 129), (32, 200), (5000, 24), (9, 70)])
def test_outputs_show_one_rounding(dtype, H, F):
    """Few neurons, many outputs of each: 11 bits of h would be a second rounding of the
    outputs that does not average out."""
    _check(Layer(2, H, F, H + F), 64, 1, dtype, seed=F)
    _check(Layer(8, H, F, H + F), 8, 4, dtype, seed=F)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("power", [1, 8, 15, 16, 17, 24, 25, 26, 28, 40])
def test_neighbours_of_far_larger_neurons(dtype, power):
    """Neurons 2^power below others of their block of 128, which no output takes."""
    H, F = 64, 192
    layer = Layer(2, H, F, power)
    # rows 128 .. 255 of both halves: neurons 128 .. 191 of g, 0 .. 63 of u
    layer.us[:, 1] *= 2.0 ** power
    layer.us *= 2.0 ** (-power / 2)
    codes = layer.down.view(torch.uint8)
    codes[:, :, :64] = 0
    codes[:, :, 128:] = 0
    _check(layer, 16, 1, dtype, seed=power)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_a_wide_range_inside_one_row_of_x(dtype):
    """Elements 2^12 to 2^26 larger than their neighbours, which half of the rows take."""
    layer = Layer(2, 256, 96, 3)
    codes = layer.up.view(torch.uint8)
    codes[:, :96, 5::16] = 0
    codes[:, 96:, 5::16] = 0

    def spoil(x):
        for i, power in enumerate((12, 20, 26)):
            x[i::3, 5::16] *= 2.0 ** power
    _check(layer, 9, 1, dtype, spoil=spoil)
    codes[:, 96:, 5::16] = 0x30
    layer.us[:, 1] *= 2.0 ** -20
    _check(layer, 9, 1, dtype, spoil=spoil)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_tiles_of_zeros_and_whole_rows_of_them(dtype):
    """Neurons that are off, and tokens without any: exact zeros."""
    need_gpu()
    layer = Layer(1, 64, 160, 1)
    layer.up.view(torch.uint8)[:, 16:48] = 0             # g of neurons 16 .. 47
    layer.up.view(torch.uint8)[:, 160 + 64:160 + 80] = 0
    ids = torch.zeros(12, 1, dtype=torch.int32, device="cuda")

    def spoil(x):
        x[3] = 0
    _check(layer, 12, 1, dtype, ids=ids, spoil=spoil)
    layer.ds *= 1e30                                     # nothing times much is nothing
    x, out = torch.zeros(2, 64, device="cuda").to(TORCH[dtype]), \
        torch.ones(2, 64, device="cuda").to(TORCH[dtype])
    layer.call(x, ids[:2], None, dtype, out)
    assert bool((out == 0).all())
