"""Outputs and inputs that are column slices of one wider buffer: the same bits as
from the same slices of buffers of their own, and nothing else of the buffer touched."""
import pytest
import torch

import all_reduce_reduction_gb300 as ar
from gpu_helpers import need_gpu
from layer_helpers import TORCH, randn

pytestmark = pytest.mark.gpu

FILL = 99.0
# widths on and off the vector paths, rows split over warps, CTAs and loops
WIDTHS = [(5, 8), (40, 130), (7, 1024), (1100, 200), (2500, 512), (3, 20001)]


class Slices:
    """Matrices of T rows of H elements side by side in one buffer (or, the same
    places, each in a buffer of its own), `gap` elements after each."""

    def __init__(self, parts, gap, together):
        T, H = parts[0].shape
        n, self.H, self.gap, self.ld = len(parts), H, gap, len(parts) * (H + gap)
        wide = [torch.full((T, self.ld), FILL, dtype=parts[0].dtype, device="cuda")
                for _ in range(1 if together else n)]
        self.wide = wide[0]
        self.at = [wide[0 if together else i][:, i * (H + gap):i * (H + gap) + H]
                   for i in range(n)]
        for v, p in zip(self.at, parts):
            v.copy_(p)

    def gaps_untouched(self):
        step = self.H + self.gap
        return all(bool((self.wide[:, i + self.H:i + step] == FILL).all())
                   for i in range(0, self.ld, step))


def _check(call, parts, gap):
    """call(slices, ld) on one buffer and on several."""
    need_gpu()
    one, several = Slices(parts, gap, True), Slices(parts, gap, False)
    extra = call(one.at, one.ld), call(several.at, several.ld)
    for i, (a, b) in enumerate(zip(one.at, several.at)):
        assert torch.equal(a, b), i
    assert all(torch.equal(a, b) for a, b in zip(*extra))
    assert one.gaps_untouched()


def _rand(seed, T, H, dtype):
    return randn(seed, T, H).to(TORCH[dtype]).cuda()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("gap", [0, 8, 3])
@pytest.mark.parametrize("T,H", WIDTHS)
def test_norm_and_gradient(dtype, gap, T, H):
    x, res, dy = (_rand(i, T, H, dtype) for i in range(3))
    g, empty = _rand(3, 1, H, dtype)[0], torch.zeros_like(x)

    def call(m, ld):
        rstd, dgamma = torch.empty(T, device="cuda"), torch.empty(H, device="cuda")
        work = torch.empty(min(T, ar.AR_NORM_GRAD_ROWS) * H, device="cuda")
        ar.ar_rmsnorm(m[0], m[2], g, 1e-6, m[1], m[3], None, rstd, T, H, dtype, ldx=ld, ldres=ld,
                      ldsum=ld, ldy=ld)
        ar.ar_rmsnorm_grad(m[4], m[0], m[1], g, rstd, m[5], dgamma, work, 4 * work.numel(), T, H,
                           dtype, lddy=ld, lddtotal=ld, ldtotal=ld, lddx=ld)
        return rstd, dgamma
    _check(call, [x, empty, res, empty, dy, empty], gap)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("gap", [0, 8, 3])
@pytest.mark.parametrize("T,H", WIDTHS)
def test_row_movers(dtype, gap, T, H):
    x, empty = _rand(1, T, H, dtype), torch.zeros(T, H, dtype=TORCH[dtype])
    row_of = torch.randperm(T, generator=torch.Generator().manual_seed(T)).int()
    row_of[T // 2] = -1
    row_of, w = row_of[:, None].cuda(), torch.rand(T, 1).cuda()

    def call(m, ld):
        dw = torch.empty(T, 1, device="cuda")
        ar.ar_moe_dispatch(m[0], None, row_of, m[1], None, T, T, 1, H, dtype, ldx=ld, ldrows=ld)
        ar.ar_moe_return(m[1], T, row_of, w, m[2], T, 1, H, dtype, ldrows=ld, ldout=ld)
        ar.ar_moe_return_grad(m[2], m[1], T, row_of, w, m[3], dw, T, 1, H, dtype, lddout=ld,
                              ldrows=ld, lddrows=ld)
        return dw,
    _check(call, [x, empty, empty, empty], gap)


@pytest.mark.parametrize("M,N,K", [(40, 64, 64), (5, 129, 512), (700, 300, 256), (33, 20, 52)])
def test_product_beside_its_operand(M, N, K):
    """a and d in one buffer of bytes: K codes (values past 448 become the NaN
    code, so the sums are compared by their bits), then N binary32 sums."""
    need_gpu()
    torch.manual_seed(293)
    ld = -(-(K + 4 * N) // 16) * 16
    codes = (torch.randn(M, K) * 100).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
    b = (torch.randn(N, K) * 100).to(torch.float8_e4m3fn).cuda()
    b = torch.nn.functional.pad(b.view(torch.uint8), (0, -K % 16))
    sa = torch.rand(M, -(-K // 128), device="cuda")
    sb = torch.rand(1, -(-N // 128), -(-K // 128), device="cuda")
    out = []
    for together in (True, False):
        wide = torch.full((M, ld), 99, dtype=torch.uint8, device="cuda")
        other = wide if together else wide.clone()
        wide[:, :K] = codes
        d = other.view(torch.float32)[:, K // 4:K // 4 + N]
        ar.ar_matmul8(wide, sa, b, sb, None, 1, d, M, N, K, "fp32", lda=ld, ldb=b.stride(0),
                      ldd=ld // 4)
        assert torch.equal(wide[:, :K], codes)
        assert bool((other[:, K + 4 * N:] == 99).all())
        out.append(d.clone().view(torch.int32))
    assert torch.equal(*out)


@pytest.mark.parametrize("H", [64, 33])
def test_one_row_in_place_has_no_stride(H):
    need_gpu()
    x, res = _rand(1, 1, H, "bf16"), _rand(2, 1, H, "bf16")
    s, y = torch.empty_like(x), torch.empty_like(x)
    ar.ar_rmsnorm(x, res, None, 1e-6, s, y, None, None, 1, H, "bf16")
    ar.ar_rmsnorm(x, res, None, 1e-6, res, x, None, None, 1, H, "bf16", ldx=H + 8, ldsum=H + 16)
    assert torch.equal(s, res) and torch.equal(y, x)


def test_rows_are_no_operand_without_dw():
    """The return's gradient does not read rows then: drows may lie across them, and
    their alignment is nothing to it."""
    need_gpu()
    T, K, H = 9, 2, 72
    dout, w = _rand(1, T, H, "bf16"), torch.rand(T, K).cuda()
    row_of = torch.randperm(T * K, generator=torch.Generator().manual_seed(1)).int().cuda()
    want = torch.zeros(T * K, H, dtype=torch.bfloat16, device="cuda")
    ar.ar_moe_return_grad(dout, None, T * K, row_of, w, want, None, T, K, H, "bf16")
    drows = torch.zeros_like(want)
    for rows in (drows.data_ptr() + 16, drows.data_ptr() + 1):
        drows.zero_()
        ar.ar_moe_return_grad(dout, rows, T * K, row_of, w, drows, None, T, K, H, "bf16")
        assert torch.equal(drows, want)
