"""ar_moe_route, ar_moe_dispatch, ar_moe_return and its gradient on the GPU.

The order, the moved rows, the fold and the rows' gradients are exact: integers,
copies, and binary32 operations in a fixed order that numpy repeats bit for bit.
dw is a sum of H products: at most H / 512 + 8 sequential adds per thread and
two trees of depth 5, within (H / 512 + 24) u of the sum of magnitudes."""
import numpy as np
import pytest
import torch

import all_reduce_reduction_gb300 as ar
from gpu_helpers import need_gpu
from layer_helpers import TORCH, U, assert_within, f64, half, placed, randn, untouched

pytestmark = pytest.mark.gpu


def _ids(T, K, E, seed, low=0, high=None):
    return np.random.default_rng(seed).integers(low, E if high is None else high, (T, K))


def _order(ids, E):
    """(offsets, row_of, src) by a stable sort."""
    flat = ids.reshape(-1)
    key = np.where((flat >= 0) & (flat < E), flat, E)
    order = np.argsort(key, kind="stable")
    row_of = np.empty(flat.size, np.int64)
    row_of[order] = np.arange(flat.size)
    offsets = np.searchsorted(key[order], np.arange(E + 1))
    return (offsets, np.where(key < E, row_of, -1).reshape(ids.shape),
            np.where(key[order] < E, order, -1))


def _route(ids, E, dtype=torch.int32, src=True):
    T, K = ids.shape
    offsets = torch.full((E + 1,), -7, dtype=torch.int32, device="cuda")
    row_of = torch.full((T, K), -7, dtype=torch.int32, device="cuda")
    s = torch.full((T * K,), -7, dtype=torch.int32, device="cuda") if src else None
    ar.ar_moe_route(torch.from_numpy(ids).to(dtype).cuda(), T, K, E, offsets, row_of, s,
                    ids_bytes=8 if dtype == torch.int64 else 4)
    return offsets, row_of, s


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("T,K,E,low,high", [
    (1, 1, 1, 0, 1), (1, 8, 64, 0, 64), (5, 3, 7, 0, 7), (16, 8, 64, 0, 64), (128, 8, 256, 0, 256),
    (129, 8, 33, 0, 33), (1000, 8, 1024, 0, 1024), (4096, 8, 64, 0, 128), (4096, 8, 64, 60, 70),
    (333, 7, 100, -50, 150), (50, 2, 8, 8, 20), (700, 32, 5, 3, 4), (70001, 3, 40, -1, 41)])
def test_route(dtype, T, K, E, low, high):
    need_gpu()
    ids = _ids(T, K, E, T + K + E, low, high)
    offsets, row_of, src = _route(ids, E, dtype)
    o, r, s = _order(ids, E)
    assert np.array_equal(offsets.cpu().numpy(), o)
    assert np.array_equal(row_of.cpu().numpy(), r)
    assert np.array_equal(src.cpu().numpy(), s)


def test_route_without_src_and_without_tokens():
    need_gpu()
    ids = _ids(40, 4, 9, 1)
    offsets, row_of, _ = _route(ids, 9, src=False)
    o, r, _ = _order(ids, 9)
    assert np.array_equal(offsets.cpu().numpy(), o) and np.array_equal(row_of.cpu().numpy(), r)
    offsets.fill_(5)
    ar.ar_moe_route(None, 0, 4, 9, offsets, None, None)
    assert bool((offsets == 0).all())


def test_route_ids_past_32_bits_are_not_here():
    need_gpu()
    ids = np.array([[1, 1 + 2 ** 32], [2 ** 40, 0], [-2 ** 33, 1]])
    offsets, row_of, src = _route(ids, 2, torch.int64)
    assert offsets.tolist() == [0, 1, 3]
    assert row_of.tolist() == [[1, -1], [-1, 0], [-1, 2]]
    assert src.tolist() == [3, 0, 5, -1, -1, -1]


SHAPES = [(1, 1, 1, 1, 0, 0), (1, 8, 16, 8192, 0, 0), (16, 8, 64, 8192, 0, 0), (9, 3, 5, 7, 0, 0),
          (33, 5, 8, 1000, 8, 0), (7, 8, 64, 4099, 0, 0), (12, 9, 32, 4099, 5, 1),
          (3, 32, 64, 130, 2, 3), (300, 2, 4, 264, 0, 0), (2, 8, 8, 20000, 0, 0)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32", "e4m3"])
@pytest.mark.parametrize("T,K,E,H,pad,shift", SHAPES)
def test_dispatch(dtype, T, K, E, H, pad, shift):
    need_gpu()
    ids = _ids(T, K, E, H + T, 0, 2 * E)                     # half of the experts elsewhere
    _, row_of, src = _order(ids, E)
    x = randn(T + H, T, H).to(torch.float32).to(TORCH[dtype])
    dx, _ = placed(x, pad, shift)
    n = T * K
    rows, buf = placed(torch.full((n, H), float("nan")).to(TORCH[dtype]), pad, shift)
    eight = dtype == "e4m3"
    nb = -(-H // 128)
    xs = torch.rand(T, nb, device="cuda") if eight else None
    rs = torch.full((n, nb), float("nan"), device="cuda") if eight else None
    ar.ar_moe_dispatch(dx, xs, torch.from_numpy(row_of).int().cuda(), rows, rs, n, T, K, H, dtype,
                       ldx=H + pad, ldrows=H + pad)
    here = int((src >= 0).sum())
    token = torch.from_numpy(src[:here] // K)
    raw = rows.cpu()
    assert torch.equal(raw[:here].float(), x.float()[token])
    assert bool(torch.isnan(raw[here:].float()).all())       # rows that no pair has
    assert untouched(buf, n, H, pad, shift)
    if eight:
        assert torch.equal(rs.cpu()[:here], xs.cpu()[token])
        assert bool(torch.isnan(rs[here:]).all())


def test_dispatch_skips_rows_past_the_buffer():
    need_gpu()
    x = randn(1, 4, 64).float().cuda()
    row_of = torch.tensor([[0, 5], [2, 9], [-3, 1], [3, 2 ** 31 - 1]], dtype=torch.int32).cuda()
    rows = torch.full((6, 64), 7.0, device="cuda")
    ar.ar_moe_dispatch(x, None, row_of, rows[:4], None, 4, 4, 2, 64, "fp32")
    assert torch.equal(rows[[0, 1, 2, 3]], x[[0, 2, 1, 3]])
    assert bool((rows[4:] == 7.0).all())


def _fold32(rows, row_of, w):
    """The fold in numpy binary32, one rounding per product and per add."""
    T, K = row_of.shape
    acc = np.zeros((T, rows.shape[1]), np.float32)
    any_ = np.zeros(T, bool)
    for k in range(K):
        at = row_of[:, k]
        here = at >= 0
        p = rows[np.maximum(at, 0)] * (w[:, k, None] if w is not None else np.float32(1))
        acc = np.where(here[:, None], np.where(any_[:, None], acc + p, p), acc)
        any_ |= here
    return acc


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("T,K,E,H,pad,shift", SHAPES)
def test_return(dtype, weighted, T, K, E, H, pad, shift):
    need_gpu()
    ids = _ids(T, K, E, H + T, 0, 2 * E)
    if T > 1:
        ids[0] = E                                           # a token without any expert here
    _, row_of, _ = _order(ids, E)
    n = T * K
    y = randn(T + H, n, H).float().to(TORCH[dtype])
    w = np.random.default_rng(T).random((T, K)).astype(np.float32) if weighted else None
    rows, _ = placed(y, pad, shift)
    out, buf = placed(torch.full((T, H), float("nan")).to(TORCH[dtype]), pad, shift)
    ar.ar_moe_return(rows, n, torch.from_numpy(row_of).int().cuda(),
                     torch.from_numpy(w).cuda() if weighted else None, out, T, K, H, dtype,
                     ldrows=H + pad, ldout=H + pad)
    y32 = y.float().numpy()
    want = torch.from_numpy(_fold32(y32, row_of, w)).to(TORCH[dtype])
    assert torch.equal(out.cpu(), want)
    if T > 1:
        assert bool((out[0] == 0).all())
    here = (row_of >= 0)[:, :, None]
    terms = y32.astype(np.float64)[np.maximum(row_of, 0)] * here
    terms = terms * (w.astype(np.float64)[:, :, None] if weighted else 1.0)
    exact = terms.sum(1)
    bound = K * U * np.abs(terms).sum(1) * (1 + 1e-6) + half(f64(out), dtype)
    assert_within(f64(out), exact, bound, "return")
    assert untouched(buf, T, H, pad, shift)


def test_return_equals_the_combine():
    """The same fold as ar_combine on rows that are in order already."""
    need_gpu()
    T, K, H = 17, 8, 2048
    rows = randn(2, K * T, H).bfloat16().cuda()
    w = torch.rand(T, K, device="cuda")
    row_of = (torch.arange(K)[None, :] * T + torch.arange(T)[:, None]).int().cuda()
    out, want = (torch.empty(T, H, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ar.ar_moe_return(rows, K * T, row_of, w, out, T, K, H, "bf16")
    with ar.Handle(K, T * H, "bf16") as h:
        ar.ar_combine(h.h, [rows[k * T:(k + 1) * T] for k in range(K)], w, want, T, H)
        assert ar.ar_status(h.h) == ar.AR_OK
    assert torch.equal(out, want)


def test_return_leaves_out_rows_elsewhere_that_hold_nan():
    need_gpu()
    rows = torch.full((4, 48), float("nan"), device="cuda")
    rows[1] = 2.0
    row_of = torch.tensor([[1, 4], [-1, 1], [7, -9]], dtype=torch.int32).cuda()
    w = torch.tensor([[0.5, float("nan")], [float("inf"), 3.0], [1.0, 1.0]], device="cuda")
    out = torch.empty(3, 48, device="cuda")
    ar.ar_moe_return(rows, 4, row_of, w, out, 3, 2, 48, "fp32")
    assert out[:, 0].tolist() == [1.0, 6.0, 0.0]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,K,E,H,pad,shift", SHAPES)
def test_return_grad(dtype, T, K, E, H, pad, shift):
    need_gpu()
    ids = _ids(T, K, E, H + T, 0, 2 * E)
    _, row_of, src = _order(ids, E)
    n = T * K
    y = randn(T + H, n, H).float().to(TORCH[dtype])
    d = randn(T + H + 1, T, H).float().to(TORCH[dtype])
    w = np.random.default_rng(T).random((T, K)).astype(np.float32)
    rows, _ = placed(y, pad, shift)
    dout, _ = placed(d, pad, shift)
    drows, buf = placed(torch.full((n, H), float("nan")).to(TORCH[dtype]), pad, shift)
    dw = torch.full((T, K), float("nan"), device="cuda")
    ar.ar_moe_return_grad(dout, rows, n, torch.from_numpy(row_of).int().cuda(),
                          torch.from_numpy(w).cuda(), drows, dw, T, K, H, dtype, lddout=H + pad,
                          ldrows=H + pad, lddrows=H + pad)
    here = int((src >= 0).sum())
    t, k = src[:here] // K, src[:here] % K
    want = torch.from_numpy(w[t, k][:, None] * d.float().numpy()[t]).to(TORCH[dtype])
    assert torch.equal(drows.cpu()[:here], want)
    assert bool(torch.isnan(drows[here:].float()).all())
    assert untouched(buf, n, H, pad, shift)
    terms = f64(d)[:, None] * f64(y)[np.maximum(row_of, 0)] * (row_of >= 0)[:, :, None]
    assert_within(f64(dw), terms.sum(2), (H / 512 + 24) * U * np.abs(terms).sum(2), "dw")


def test_return_grad_against_differences():
    """The fold is linear in the rows and in the weights, so differences of the
    binary64 forward are exact up to its rounding."""
    need_gpu()
    T, K, E, H = 3, 2, 4, 24
    _, row_of, _ = _order(_ids(T, K, E, 5), E)
    y, d = randn(6, T * K, H).float(), randn(7, T, H).float()
    w = torch.rand(T, K, generator=torch.Generator().manual_seed(8))
    drows, dw = torch.zeros(T * K, H, device="cuda"), torch.empty(T, K, device="cuda")
    ar.ar_moe_return_grad(d.cuda(), y.cuda(), T * K, torch.from_numpy(row_of).int().cuda(),
                          w.cuda(), drows, dw, T, K, H, "fp32")

    def loss(rows, weights):
        return ((weights[:, :, None] * rows[row_of]).sum(1) * f64(d)).sum()
    y64, w64, h = f64(y), f64(w), 0.5
    for r, i in [(0, 0), (3, 11), (5, 23)]:
        step = np.zeros_like(y64)
        step[r, i] = h
        assert abs(float(drows[r, i]) - (loss(y64 + step, w64) - loss(y64 - step, w64)) / (2 * h)) \
            <= 1e-6
    for t, k in [(0, 0), (2, 1)]:
        step = np.zeros_like(w64)
        step[t, k] = h
        assert abs(float(dw[t, k]) - (loss(y64, w64 + step) - loss(y64, w64 - step)) / (2 * h)) \
            <= 2e-5


def test_return_grad_parts_and_in_place():
    need_gpu()
    T, K, E, H = 21, 8, 16, 1032
    _, row_of, _ = _order(_ids(T, K, E, 3), E)
    row_of = torch.from_numpy(row_of).int().cuda()
    rows, dout = randn(4, T * K, H).bfloat16().cuda(), randn(5, T, H).bfloat16().cuda()
    w = torch.rand(T, K, device="cuda")
    drows, dw = torch.empty_like(rows), torch.empty(T, K, device="cuda")
    ar.ar_moe_return_grad(dout, rows, T * K, row_of, w, drows, dw, T, K, H, "bf16")
    only, only_dw = torch.empty_like(rows), torch.empty_like(dw)
    ar.ar_moe_return_grad(dout, None, T * K, row_of, w, only, None, T, K, H, "bf16")
    ar.ar_moe_return_grad(dout, rows, T * K, row_of, w, None, only_dw, T, K, H, "bf16")
    assert torch.equal(only, drows) and torch.equal(only_dw, dw)
    ar.ar_moe_return_grad(dout, rows, T * K, row_of, w, rows, only_dw, T, K, H, "bf16")
    assert torch.equal(rows, drows) and torch.equal(only_dw, dw)


def test_dispatch_gradient_is_the_unweighted_return():
    """<dispatch(x), r> = <x, return(r)> with integers, where both are exact."""
    need_gpu()
    T, K, E, H = 13, 4, 6, 200
    _, row_of, _ = _order(_ids(T, K, E, 9, 0, 9), E)
    row_of = torch.from_numpy(row_of).int().cuda()
    g = torch.Generator().manual_seed(1)
    x = torch.randint(-8, 9, (T, H), generator=g).float().cuda()
    r = torch.randint(-8, 9, (T * K, H), generator=g).float().cuda()
    rows, out = torch.zeros(T * K, H, device="cuda"), torch.empty(T, H, device="cuda")
    ar.ar_moe_dispatch(x, None, row_of, rows, None, T * K, T, K, H, "fp32")
    ar.ar_moe_return(r, T * K, row_of, None, out, T, K, H, "fp32")
    assert float((rows.double() * r.double()).sum()) == float((x.double() * out.double()).sum())


def test_row_movers_without_tokens_or_rows():
    need_gpu()
    out = torch.full((2, 8), 5.0, device="cuda")
    row_of = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    ar.ar_moe_dispatch(None, None, None, out, None, 2, 0, 1, 8, "fp32")
    ar.ar_moe_return(None, 0, None, None, None, 0, 1, 8, "fp32")
    assert bool((out == 5.0).all())
    ar.ar_moe_return(None, 0, row_of, None, out, 2, 1, 8, "fp32")      # no rows: zeros
    assert bool((out == 0.0).all())


def test_the_path_in_a_graph():
    """Route, dispatch and return captured together, replayed on other ids."""
    need_gpu()
    T, K, E, H = 64, 8, 32, 512
    x = randn(1, T, H).bfloat16().cuda()
    w = torch.rand(T, K, device="cuda")
    ids = torch.zeros(T, K, dtype=torch.int32, device="cuda")
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    row_of = torch.zeros(T, K, dtype=torch.int32, device="cuda")
    rows = torch.zeros(T * K, H, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")

    def path(stream):
        ar.ar_moe_route(ids, T, K, E, offsets, row_of, None, stream=stream)
        ar.ar_moe_dispatch(x, None, row_of, rows, None, T * K, T, K, H, "bf16", stream=stream)
        ar.ar_moe_return(rows, T * K, row_of, w, out, T, K, H, "bf16", stream=stream)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        path(s)
    for seed in (1, 2):
        new = _ids(T, K, E, seed)
        ids.copy_(torch.from_numpy(new).int())
        g.replay()
        torch.cuda.synchronize()
        _, r, _ = _order(new, E)
        assert np.array_equal(row_of.cpu().numpy(), r)
        y = x.float().cpu().numpy()
        want = _fold32(np.repeat(y, K, 0), np.arange(T * K).reshape(T, K), w.cpu().numpy())
        assert torch.equal(out.cpu(), torch.from_numpy(want).bfloat16())
