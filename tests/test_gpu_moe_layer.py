"""ar_moe_layer on the GPU against the definition in binary64.

Bound.  A block's 128 products are exact in binary32 and summed by a tensor core in eight
steps of 16 terms, each of which may lose 4 u of the magnitudes (u = 2^-24); twice that where
x or h has two parts: 64 u.  Scales, joining the blocks and the warps' sums: 6 u a block and
one more per addition.  With a = (80 + 2 blocks) u:
  |dg| <= a sum |up||x|,  likewise u
  |dh| <= 1.1 |u| |dg| + |silu(g)| |du| + 16 u |h|     (the slope of silu is below 1.1)
  |dy| <= sum |down| (|dh| + r |h|) + a' sum |down||h|
x in binary32 has two parts of 11 bits, 2^-21 of x, and so has h then (r = 2^-21); for
outputs of two bytes h has one, off by half a unit of binary16: r = 2^-11.  What lies more
than 2^-29 below a block's largest element is a subnormal there, off by 2^-25 where the
largest is at least 2^14: 2^-39 of it.  Then the weighted sum over the choices, and one
rounding to the output."""
import pytest
import torch

import all_reduce_reduction_gb300 as ar
from gpu_helpers import need_gpu
from layer_helpers import TORCH, U, assert_within, half, untouched

pytestmark = pytest.mark.gpu


def _codes(g, E, rows, K, pad, shift=0):
    v = (torch.randn(E * rows, K, generator=g, device="cuda") * 100).clamp(-448, 448)
    buf = torch.full((shift + E * rows * (K + pad),), 0x7F, dtype=torch.uint8, device="cuda")
    view = buf[shift:].view(E * rows, K + pad)[:, :K]
    view.copy_(v.to(torch.float8_e4m3fn).view(torch.uint8))
    return view.view(torch.float8_e4m3fn).unflatten(0, (E, rows))


class Layer:
    def __init__(self, E, H, F, seed=0, pad=None, shift=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.E, self.H, self.F = E, H, F
        pads = ((-H) % 16, (-F) % 16) if pad is None else (pad, pad)
        self.up, self.down = _codes(g, E, 2 * F, H, pads[0], shift), _codes(g, E, H, F, pads[1],
                                                                          shift)
        self.ld = H + pads[0], F + pads[1]

        def scales(rows, cols):
            r = torch.rand(E, -(-rows // 128), -(-cols // 128), generator=g, device="cuda")
            return (0.5 + r) * (cols ** -0.5 / 100)
        self.us, self.ds = scales(2 * F, H), scales(H, F)

    def call(self, x, ids, w, dtype, out, ldx=0, ldout=0, stream=None):
        T, K = ids.shape
        work = torch.full((T * K * (self.F + 128),), float("nan"), device="cuda")
        ar.ar_moe_layer(x, ids, w, self.up, self.us, self.down, self.ds, out, work,
                        4 * work.numel(), T, K, self.E, self.H, self.F, dtype, ldx=ldx,
                        ldup=self.ld[0], lddown=self.ld[1], ldout=ldout, stream=stream)
        return work

    def exact(self, x, ids, w, dtype):
        """(out, bound without the output's rounding) in binary64."""
        T, K = ids.shape
        H, F = self.H, self.F
        hb, fb = -(-H // 128), -(-F // 128)
        i = {n: torch.arange(n, device="cuda") // 128 for n in (H, F, 2 * F)}
        out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        err, size = torch.zeros_like(out), torch.zeros_like(out)
        a1, a2 = (80 + 2 * hb) * U, (80 + 2 * fb) * U
        if dtype == "fp32":
            a1 += 2.0 ** -21
        for e in sorted(set(ids.flatten().tolist())):
            if not 0 <= e < self.E:
                continue
            t, k = torch.nonzero(ids == e, as_tuple=True)
            w1 = self.up[e].float().double() * self.us[e].double()[i[2 * F]][:, i[H]]
            w2 = self.down[e].float().double() * self.ds[e].double()[i[H]][:, i[F]]
            v = x[t].double()
            both, mag = v @ w1.t(), v.abs() @ w1.abs().t()
            mag = a1 * mag + 2.0 ** -39 * v.abs().amax(1, keepdim=True) * w1.abs().sum(1)
            g, u = both.split(F, 1)
            dg, du = mag.split(F, 1)
            act = g * torch.sigmoid(g)
            h = act * u
            dh = 1.1 * (u.abs() + du) * dg + act.abs() * du + 16 * U * h.abs()
            y = h @ w2.t()
            off = 2.0 ** (-21 if dtype == "fp32" else -11)
            dy = (dh + off * h.abs()) @ w2.abs().t() + a2 * (h.abs() @ w2.abs().t())
            dy += 2.0 ** -39 * h.abs().amax(1, keepdim=True) * w2.abs().sum(1)
            gate = torch.ones(len(t), 1, dtype=torch.float64, device="cuda") if w is None else \
                w[t, k, None].double()
            out.index_add_(0, t, gate * y)
            err.index_add_(0, t, gate.abs() * dy)
            size.index_add_(0, t, gate.abs() * (h.abs() @ w2.abs().t()))
        return out, err + (K + 10) * U * size


def _ids(T, K, E, seed, total=None, dtype=torch.int32):
    """K different experts a token, of `total` (those past E are elsewhere)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    score = torch.rand(T, max(total or E, K), generator=g, device="cuda")
    return torch.topk(score, K, dim=1).indices.to(dtype)


def _check(T, K, E, H, F, dtype, total=None, ids=None, weights=True, xpad=0, seed=0, pad=None,
           shift=0, x_std=1.0, ids_dtype=torch.int32, layer=None):
    need_gpu()
    layer = layer or Layer(E, H, F, seed, pad, shift)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    buf = torch.full((T, H + xpad), float("nan"), device="cuda").to(TORCH[dtype])
    x = buf[:, :H]
    x.copy_(x_std * torch.randn(T, H, generator=g, device="cuda"))
    if ids is None:
        ids = _ids(T, K, E, seed + 2, total, ids_dtype)
    else:
        ids = torch.tensor(ids, dtype=ids_dtype, device="cuda").view(T, K)
    w = torch.rand(T, K, generator=g, device="cuda") if weights else None
    obuf = torch.full((T, H + xpad), float("nan"), device="cuda").to(TORCH[dtype])
    layer.call(x, ids, w, dtype, obuf, ldx=H + xpad, ldout=H + xpad)
    torch.cuda.synchronize()
    want, err = layer.exact(x.float(), ids, w, dtype)
    want, err = want.cpu().numpy(), err.cpu().numpy()
    assert untouched(obuf.view(-1), T, H, xpad, 0)
    assert_within(obuf[:, :H].double().cpu().numpy(), want, err + half(want, dtype) * (1 + 1e-6),
                  "out")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,K,E,H,F", [
    (1, 1, 1, 1, 1), (1, 1, 1, 16, 16), (1, 2, 4, 128, 128), (1, 8, 64, 512, 256), (2, 3, 5, 100, 70),
    (3, 1, 2, 1000, 33), (4, 2, 8, 1000, 520), (7, 2, 3, 129, 257), (8, 2, 2, 256, 640),
    (9, 1, 1, 384, 130), (16, 4, 8, 640, 384), (17, 2, 2, 144, 100), (33, 1, 1, 200, 72),
    (64, 1, 2, 272, 144), (64, 8, 64, 512, 128), (64, 8, 8, 130, 96), (16, 32, 40, 128, 64),
    (1, 1, 1, 8192, 64), (1, 2, 3, 64, 4000), (5, 3, 1000, 32, 16)])
def test_sizes(dtype, T, K, E, H, F):
    _check(T, K, E, H, F, dtype, seed=T + H)


@pytest.mark.parametrize("T,K,E,H,F,pad,shift,xpad", [
    (3, 2, 4, 200, 90, 0, 0, 0), (3, 2, 4, 200, 90, 5, 0, 3), (2, 2, 4, 256, 128, 0, 1, 0),
    (4, 1, 2, 256, 128, 16, 16, 8), (4, 1, 2, 240, 112, 0, 0, 1), (9, 2, 3, 257, 129, 1, 3, 5)])
def test_strides_and_alignment(T, K, E, H, F, pad, shift, xpad):
    for dtype in ("bf16", "fp32"):
        _check(T, K, E, H, F, dtype, pad=pad, shift=shift, xpad=xpad, seed=H)


@pytest.mark.parametrize("ids", [
    [[-1, -1], [9, 100]], [[0, 0], [0, 0]], [[1, 1], [-1, 1]], [[3, 2], [2, 3]],
    [[2 ** 31 - 1, -2 ** 31], [0, 3]], [[3, 3], [3, -5]]], ids=str)
@pytest.mark.parametrize("ids_dtype", [torch.int32, torch.int64])
def test_choices(ids, ids_dtype):
    """None here, one expert for all, a token that names an expert twice, ids out of range."""
    _check(2, 2, 4, 136, 72, "fp32", ids=ids, ids_dtype=ids_dtype)


def test_ids_beyond_32_bits_are_elsewhere():
    _check(2, 2, 4, 64, 32, "fp32", ids=[[2 ** 32, 1], [2 ** 40 + 1, -2 ** 33]],
           ids_dtype=torch.int64)


@pytest.mark.parametrize("T", [1, 8, 9, 31, 32, 33, 40, 64])
def test_every_token_to_one_expert(T):
    """More pairs of an expert than one pass over its weights holds."""
    _check(T, 2, 3, 144, 80, "bf16", ids=[[1, 1 if t % 3 else 0] for t in range(T)])
    _check(T, 4, 6, 100, 40, "fp32", ids=[[5, 5, 5, 5]] * T)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_without_weights_and_with_experts_elsewhere(dtype):
    _check(6, 4, 8, 256, 144, dtype, total=32, weights=False)
    _check(6, 4, 8, 256, 144, dtype, total=16)


def test_large_and_small_inputs():
    """Inputs whose magnitudes lie outside binary16, and a wide range inside one row."""
    for std in (1e-30, 1e-8, 1e6, 1e15):
        layer = Layer(2, 256, 128, 3)
        layer.us.mul_(1 / std)
        _check(3, 2, 2, 256, 128, "bf16", x_std=std, layer=layer)
        _check(3, 2, 2, 256, 128, "fp32", x_std=std, layer=layer)


def test_nan_and_infinities_stay_with_their_token():
    need_gpu()
    layer = Layer(3, 256, 128)
    x = torch.randn(5, 256, device="cuda").bfloat16()
    ids = torch.tensor([[0, 1], [1, 2], [2, 0], [0, 2], [1, 0]], dtype=torch.int32, device="cuda")
    w = torch.rand(5, 2, device="cuda")
    clean, out = torch.empty_like(x), torch.empty_like(x)
    layer.call(x, ids, w, "bf16", clean)
    x[1, 7], x[3, 200] = float("nan"), float("inf")
    layer.call(x, ids, w, "bf16", out)
    assert not bool(torch.isfinite(out[1]).any()) and not bool(torch.isfinite(out[3]).any())
    keep = torch.tensor([0, 2, 4], device="cuda")
    assert torch.equal(out[keep], clean[keep])
    # a NaN weight of an expert reaches the tokens that chose it
    layer.down.view(torch.uint8)[1, 30, 5] = 0x7F
    x[1, 7], x[3, 200] = 0.0, 0.0
    layer.call(x, ids, w, "bf16", out)
    assert bool(torch.isnan(out[torch.tensor([0, 1, 4], device="cuda"), 30]).all())
    assert torch.equal(out[2], clean[2]) and bool(torch.isfinite(out[3]).all())


def test_same_bits_every_time_and_in_a_graph():
    """One capture serves any choices: they are read on the device."""
    need_gpu()
    T, K, E, H, F = 6, 3, 16, 512, 256
    layer = Layer(E, H, F)
    x = torch.randn(T, H, device="cuda").bfloat16()
    ids, w = _ids(T, K, E, 0), torch.rand(T, K, device="cuda")
    out, once = torch.empty_like(x), torch.empty_like(x)
    work = torch.empty(T * K * (F + 128), device="cuda")
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        ar.ar_moe_layer(x, ids, w, layer.up, layer.us, layer.down, layer.ds, out, work,
                        4 * work.numel(), T, K, E, H, F, "bf16", stream=s)
    for seed in range(4):
        ids.copy_(_ids(T, K, E, seed, total=E if seed else 4 * E))
        layer.call(x, ids, w, "bf16", once)
        for _ in range(5):
            out.fill_(3)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, once)


def test_zero_tokens():
    need_gpu()
    layer = Layer(2, 64, 32)
    ar.ar_moe_layer(None, None, None, layer.up, layer.us, layer.down, layer.ds, None, None, 0, 0, 2,
                    2, 64, 32, "bf16", ids_bytes=4)
    torch.cuda.synchronize()


def test_against_the_call_by_call_layer():
    """What the dispatch, the products and the return make of the same weights, but for
    the 8-bit rounding of what goes into the products: 2^-4 of an element at most."""
    need_gpu()
    T, K, E, H, F = 24, 2, 4, 512, 256
    layer, n = Layer(E, H, F), 24 * 2
    x = torch.randn(T, H, device="cuda").bfloat16()
    ids, w = _ids(T, K, E, 5), torch.rand(T, K, device="cuda")
    out = torch.empty_like(x)
    layer.call(x, ids, w, "bf16", out)
    i32, f8 = dict(dtype=torch.int32, device="cuda"), dict(dtype=torch.float8_e4m3fn, device="cuda")
    offsets, row_of = torch.empty(E + 1, **i32), torch.empty(T, K, **i32)

    def eight(v):
        q, s = torch.empty(v.shape, **f8), torch.empty(v.shape[0], v.shape[1] // 128, device="cuda")
        b = v.float().unflatten(1, (-1, 128))
        s.copy_(b.abs().amax(2) / 448)
        q.copy_((b / s[:, :, None]).flatten(1))
        return q, s
    q, s = eight(x)
    rows, rs = torch.zeros(n, H, **f8), torch.zeros(n, H // 128, device="cuda")
    ar.ar_moe_route(ids, T, K, E, offsets, row_of)
    ar.ar_moe_dispatch(q, s, row_of, rows, rs, n, T, K, H, "e4m3")
    both, y, other = torch.empty(n, 2 * F, device="cuda"), torch.empty(n, H, device="cuda"), \
        torch.empty(T, H, device="cuda")
    ar.ar_matmul8(rows, rs, layer.up, layer.us, offsets, E, both, n, 2 * F, H, "fp32")
    g, u = both.chunk(2, 1)
    ar.ar_matmul8(*eight(torch.nn.functional.silu(g) * u), layer.down, layer.ds, offsets, E, y, n,
                  H, F, "fp32")
    ar.ar_moe_return(y, n, row_of, w, other, T, K, H, "fp32")
    assert float((out.float() - other).norm() / other.norm()) < 2 ** -4
