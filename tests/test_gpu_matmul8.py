"""ar_matmul8 on the GPU against the definition in binary64.

Bound.  E4M3 products are exact in binary32.  A block's 128 products are summed
in binary32; a tensor core aligns the terms of a step to the largest before it
adds them and may cut what lies below its accumulator's last bits, so a step's
error is taken as at most 4 units of 2^-24 of the magnitudes in it, and eight
such steps (of 16 or 32 terms) make a block: 32 u of the block's sum of
magnitudes.  Scaling and joining the blocks adds 3 u per block and one u per
add, at most (3 + blocks) u of the same sum.  Then one rounding to the output."""
import numpy as np
import pytest
import torch

import all_reduce_reduction_gb300 as ar
from gpu_helpers import need_gpu
from layer_helpers import TORCH, U, assert_within, half, untouched

pytestmark = pytest.mark.gpu


def _codes(seed, rows, K, pad, shift=0):
    """E4M3 rows with `pad` bytes of NaN codes after each and `shift` before."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = (torch.randn(rows, K, generator=g, device="cuda") * 100).clamp(-448, 448)
    buf = torch.full((shift + rows * (K + pad),), 0x7F, dtype=torch.uint8, device="cuda")
    view = buf[shift:].view(rows, K + pad)[:, :K]
    view.copy_(v.to(torch.float8_e4m3fn).view(torch.uint8))
    return view.view(torch.float8_e4m3fn)


def _scales(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand(*shape, generator=g, device="cuda") * 0.02 + 1e-4


def _exact(a, sa, b, sb, offsets):
    """(d, sum of magnitudes) in binary64, group by group; NaN where no group has the row."""
    M, K = a.shape
    E, N = b.shape[:2]
    kb = torch.arange(K, device="cuda") // 128
    nb = torch.arange(N, device="cuda") // 128
    a64 = a.float().double() * sa.double()[:, kb]
    d = torch.full((M, N), float("nan"), dtype=torch.float64, device="cuda")
    size = torch.zeros_like(d)
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        b64 = b[e].float().double() * sb[e].double()[nb][:, kb]
        d[lo:hi] = a64[lo:hi] @ b64.t()
        size[lo:hi] = a64[lo:hi].abs() @ b64.abs().t()
    return d.cpu().numpy(), size.cpu().numpy()


def _run(M, N, K, out, offsets=None, pad=None, shift=0, ldd_pad=0, seed=0, spoil=None):
    """offsets: a list, or None for one matrix.  pad None: rows 16-byte aligned."""
    need_gpu()
    E = 1 if offsets is None else len(offsets) - 1
    pad = (-K) % 16 if pad is None else pad
    kb, nb = -(-K // 128), -(-N // 128)
    a = _codes(seed + 1, M, K, pad, shift)
    b = _codes(seed + 2, E * N, K, pad, shift).unflatten(0, (E, N))
    sa, sb = _scales(seed + 3, M, kb), _scales(seed + 4, E, nb, kb)
    if spoil is not None:
        spoil(a, sa, b, sb)
    buf = torch.full((M * (N + ldd_pad),), float("nan"), device="cuda").to(TORCH[out])
    d = buf.view(M, N + ldd_pad)[:, :N]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    ar.ar_matmul8(a, sa, b, sb, off, E, d, M, N, K, out, lda=K + pad, ldb=K + pad,
                  ldd=N + ldd_pad, status=status)
    torch.cuda.synchronize()
    assert int(status) == ar.AR_OK
    assert untouched(buf, M, N, ldd_pad, 0)
    return a, sa, b, sb, d


def _check(M, N, K, out, offsets=None, **kw):
    a, sa, b, sb, d = _run(M, N, K, out, offsets, **kw)
    want, size = _exact(a, sa, b, sb, [0, M] if offsets is None else offsets)
    got = d.float().double().cpu().numpy()
    none = np.isnan(want)
    assert np.isnan(got[none]).all()                         # rows of no group
    got, want, size = got[~none], want[~none], size[~none]
    bound = (35 + -(-K // 128)) * U * size + half(want, out) * (1 + 1e-6)
    if out == "fp16":
        bound = bound + np.where(np.abs(want) > 65000, np.inf, 0)
    assert_within(got, want, bound, "d")


@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 1), (1, 128, 128), (3, 5, 7), (1, 1000, 200), (1, 8192, 1024), (2, 129, 257),
    (16, 256, 512), (17, 300, 144), (33, 640, 1000), (64, 2048, 256), (100, 384, 4096),
    (128, 256, 128), (129, 257, 129), (255, 513, 640), (256, 1024, 2048), (300, 100, 100),
    (1000, 776, 520), (2048, 2048, 384), (2500, 2600, 130), (4096, 1100, 1000), (129, 40000, 256),
    (33000, 40, 64)])
def test_one_matrix(M, N, K, out):
    _check(M, N, K, out, seed=M + N + K)


@pytest.mark.parametrize("M,N,K,pad,shift,ldd_pad", [
    (5, 70, 100, 0, 0, 0), (70, 130, 131, 0, 0, 3), (33, 200, 256, 1, 0, 0), (40, 96, 128, 0, 5, 1),
    (130, 140, 300, 20, 0, 7), (300, 260, 200, 24, 16, 5), (200, 300, 128, 0, 0, 1)])
def test_strides_and_alignment(M, N, K, pad, shift, ldd_pad):
    _check(M, N, K, "fp32", pad=pad, shift=shift, ldd_pad=ldd_pad, seed=M)
    _check(M, N, K, "bf16", pad=pad, shift=shift, ldd_pad=ldd_pad, seed=M + 1)


GROUPS = [
    [0, 0, 0, 5], [0, 1, 2, 3, 4, 5, 6, 7, 8], [0, 64, 64, 100, 300], [0, 128, 256, 400],
    [0, 130, 130, 131, 500], [7, 20, 20, 90], [0, 0], [3, 3, 3], [0, 17, 34, 51, 700, 701],
    [0, 300, 900, 901, 1700]]


@pytest.mark.parametrize("offsets", GROUPS, ids=lambda o: "-".join(map(str, o)))
@pytest.mark.parametrize("N,K", [(256, 256), (200, 400), (1030, 136)])
def test_groups(offsets, N, K):
    """Empty groups, groups that end inside a tile, rows of no group on both ends."""
    _check(offsets[-1] + 9, N, K, "bf16", offsets, seed=N)


@pytest.mark.parametrize("N,K", [(1500, 400), (513, 1024)])
def test_groups_of_a_prefill(N, K):
    """Enough tiles for every SM: uneven groups, some empty, columns ragged."""
    rng = np.random.default_rng(N)
    counts = np.where(rng.random(60) < 0.2, 0, rng.integers(1, 700, 60))
    offsets = [0] + np.cumsum(counts).tolist()
    _check(offsets[-1] + 200, N, K, "bf16", offsets, seed=N, ldd_pad=N % 2 * 3)


def test_groups_without_alignment():
    _check(150, 131, 133, "fp32", [2, 2, 60, 61, 140], pad=0, seed=2)


def test_many_groups():
    rng = np.random.default_rng(3)
    counts = rng.integers(0, 9, 300)
    offsets = [0] + np.cumsum(counts).tolist()
    _check(offsets[-1] + 1, 144, 160, "bf16", offsets, seed=9)


def test_offsets_outside_the_rows_count_as_the_ends():
    a, sa, b, sb, d = _run(50, 64, 64, "fp32", [-5, 20, 2 ** 31 - 1], seed=4)
    want, size = _exact(a, sa, b, sb, [0, 20, 50])
    assert_within(d.double().cpu().numpy(), want, 40 * U * size + half(want, "fp32"), "d")


@pytest.mark.parametrize("M", [40, 400])
def test_nan_codes_and_infinite_scales_stay_in_their_rows(M):
    """A NaN code spoils its row, a NaN weight its column, an infinite scale its
    row; every other element is as it would be."""
    offsets = [0, M // 2, M]
    clean = _run(M, 300, 272, "fp32", offsets, seed=5)[4]

    def spoil(a, sa, b, sb):
        a.view(torch.uint8)[M // 2 - 1, 100] = 0x7F
        b.view(torch.uint8)[1, 70, 3] = 0x7F
        sa[M - 2, 1] = float("inf")
    d = _run(M, 300, 272, "fp32", offsets, seed=5, spoil=spoil)[4]
    bad = torch.zeros(M, 300, dtype=torch.bool, device="cuda")
    bad[M // 2 - 1] = True
    bad[M // 2:, 70] = True
    assert bool(torch.isnan(d[bad]).all())
    bad[M - 2] = True
    assert bool((~torch.isfinite(d[M - 2])).all())
    assert torch.equal(d[~bad], clean[~bad])


def test_zero_rows():
    need_gpu()
    d = torch.full((1, 64), 3.0, device="cuda")
    b = _codes(1, 64, 64, 0)[None]
    ar.ar_matmul8(None, None, b, _scales(2, 1, 1, 1), None, 1, d, 0, 64, 64, "fp32")
    torch.cuda.synchronize()
    assert bool((d == 3.0).all())


@pytest.mark.parametrize("M", [24, 600, 20000])
def test_in_a_graph_with_other_offsets(M):
    """One capture serves any grouping: the offsets are read on the device."""
    need_gpu()
    E, N, K = 4, 256, 384
    a, b = _codes(1, M, K, 0), _codes(2, E * N, K, 0).unflatten(0, (E, N))
    sa, sb = _scales(3, M, 3), _scales(4, E, 2, 3)
    d = torch.zeros(M, N, device="cuda")
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        ar.ar_matmul8(a, sa, b, sb, off, E, d, M, N, K, "fp32", stream=s)
    for cuts in ([0, M // 3, M // 2, M // 2, M], [0, 0, 1, M - 1, M]):
        off.copy_(torch.tensor(cuts, dtype=torch.int32))
        d.zero_()
        g.replay()
        torch.cuda.synchronize()
        want, size = _exact(a, sa, b, sb, cuts)
        assert_within(d.double().cpu().numpy(), want, 40 * U * size + half(want, "fp32"), "d")
