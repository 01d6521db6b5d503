"""Buffers past 4 GiB: byte offsets that do not fit 32 bits, in every layer
operator.  The check is on rows at both ends and around the 4 GiB mark."""
import numpy as np
import pytest
import torch

import all_reduce_reduction_gb300 as ar
from gpu_helpers import need_gpu
from layer_helpers import U, assert_within, f64, half

pytestmark = pytest.mark.gpu
H = 8192
ROWS = (1 << 32) // (2 * H) + 1500           # bf16 rows: 4 GiB and some


def _probe(n):
    mark = (1 << 32) // (2 * H)
    return torch.tensor([0, 1, mark - 1, mark, mark + 1, n - 2, n - 1])


def _fill(n, k=H, dtype=torch.bfloat16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.empty(n, k, dtype=torch.bfloat16, device="cuda").normal_(0, 1, generator=g)
    return x if dtype is torch.bfloat16 else (x.clamp_(-4, 4) * 100).to(dtype)


def test_norm_and_gradient():
    need_gpu()
    x = _fill(ROWS)
    s, y = torch.empty_like(x), torch.empty_like(x)
    rstd = torch.empty(ROWS, device="cuda")
    ar.ar_rmsnorm(x, x, None, 1e-6, s, y, None, rstd, ROWS, H, "bf16")
    at = _probe(ROWS).cuda()
    v = 2 * f64(x[at])
    want = v / np.sqrt((v * v).mean(1, keepdims=True) + 1e-6)
    assert torch.equal(s[at].float(), 2 * x[at].float())
    assert_within(f64(y[at]), want, 64 * U * np.abs(want) + half(want, "bf16"), "y")
    dx = torch.empty_like(x)
    ar.ar_rmsnorm_grad(y, None, s, None, rstd, dx, None, None, 0, ROWS, H, "bf16")
    n, d, r = f64(s[at]) * f64(rstd[at])[:, None], f64(y[at]), f64(rstd[at])[:, None]
    inner = (d * n).mean(1, keepdims=True)
    size = r * (np.abs(d) + np.abs(n) * np.abs(d * n).mean(1, keepdims=True))
    want = r * (d - n * inner)
    assert_within(f64(dx[at]), want, 96 * U * size + half(want, "bf16"), "dx")


def test_row_movers():
    need_gpu()
    T, K = ROWS // 4, 4
    n = T * K
    ids = torch.arange(n, dtype=torch.int32, device="cuda").view(T, K) % 7
    offsets = torch.empty(8, dtype=torch.int32, device="cuda")
    row_of = torch.empty(T, K, dtype=torch.int32, device="cuda")
    src = torch.empty(n, dtype=torch.int32, device="cuda")
    ar.ar_moe_route(ids, T, K, 7, offsets, row_of, src)
    x = _fill(T, seed=1)
    rows = torch.empty(n, H, dtype=torch.bfloat16, device="cuda")
    ar.ar_moe_dispatch(x, None, row_of, rows, None, n, T, K, H, "bf16")
    at = _probe(n).cuda()
    assert torch.equal(rows[at], x[src[at].long() // K])
    out = torch.empty_like(x)
    ar.ar_moe_return(rows, n, row_of, None, out, T, K, H, "bf16")
    assert torch.equal(out[-3:].float(), 4 * x[-3:].float())
    w = torch.rand(T, K, device="cuda")
    drows, dw = torch.empty_like(rows), torch.empty(T, K, device="cuda")
    ar.ar_moe_return_grad(x, rows, n, row_of, w, drows, dw, T, K, H, "bf16")
    pair = src[at].long()
    want = (w.view(-1)[pair, None] * x[pair // K].float()).bfloat16()
    assert torch.equal(drows[at], want)
    d = f64(x[-2:])
    exact = np.repeat((d * d).sum(1)[:, None], K, 1)
    assert_within(f64(dw[-2:]), exact, (H / 512 + 24) * U * exact, "dw")


@pytest.mark.parametrize("N", [16, 512])
def test_matmul8(N):
    need_gpu()
    K = H
    M = (1 << 32) // K + 777                    # bytes of a past 4 GiB
    a, b = _fill(M, K, torch.float8_e4m3fn, 2), _fill(N, K, torch.float8_e4m3fn, 3)
    sa = torch.rand(M, K // 128, device="cuda") * 0.01
    sb = torch.rand(1, -(-N // 128), K // 128, device="cuda") * 0.01
    d = torch.empty(M, N, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ar.ar_matmul8(a, sa, b, sb, None, 1, d, M, N, K, "fp32", status=status)
    torch.cuda.synchronize()
    assert int(status) == ar.AR_OK
    mark = (1 << 32) // K
    at = torch.tensor([0, 1, mark - 1, mark, mark + 1, M - 2, M - 1], device="cuda")
    kb = torch.arange(K, device="cuda") // 128
    nb = torch.arange(N, device="cuda") // 128
    codes = a.view(torch.uint8)[at].view(torch.float8_e4m3fn)
    a64 = codes.float().double() * sa[at].double()[:, kb]
    b64 = b.float().double() * sb[0].double()[nb][:, kb]
    want, size = (a64 @ b64.t()).cpu().numpy(), (a64.abs() @ b64.abs().t()).cpu().numpy()
    assert_within(d[at].double().cpu().numpy(), want, (35 + K // 128) * U * size
                  + half(want, "fp32"), "d")
