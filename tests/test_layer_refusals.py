"""What the layer operators refuse, each before any CUDA call (so these run
without a GPU; the addresses are never dereferenced)."""
import pytest

import all_reduce_reduction_gb300 as ar
from all_reduce_reduction_gb300 import build as cuda_build

A = [0x10000000 * (i + 1) for i in range(10)]       # distinct 16-byte aligned addresses
INVALID, UNSUPPORTED = ar.AR_ERR_INVALID, ar.AR_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def built():
    cuda_build.build()


def _code(fn, *args, **kw):
    try:
        fn(*args, stream=0, **kw)
    except ar.ArError as e:
        return e.code
    return ar.AR_OK


def _norm(**kw):
    a = dict(x=A[0], res=A[1], gamma=A[2], eps=1e-6, total=A[3], y=A[4], scale=None, rstd=A[5],
             T=4, H=256, dtype="bf16", out_dtype=None)
    a.update(kw)
    return _code(ar.ar_rmsnorm, **a)


@pytest.mark.parametrize("change", [
    dict(x=None), dict(y=None), dict(H=0), dict(dtype=8), dict(dtype=3), dict(out_dtype="fp32"),
    dict(out_dtype="e4m3"), dict(scale=A[6]), dict(eps=-1.0), dict(eps=float("nan")),
    dict(x=A[0] + 1), dict(res=A[1] + 1), dict(gamma=A[2] + 1), dict(total=A[3] + 1),
    dict(rstd=A[5] + 2), dict(ldx=255), dict(ldres=1), dict(ldsum=255), dict(ldy=200),
    dict(y=A[3]), dict(y=A[3] + 512), dict(total=A[0] + 512), dict(y=A[1] + 2), dict(y=A[2]),
    dict(total=A[2]), dict(rstd=A[4] + 16), dict(rstd=A[0]), dict(total=A[0], y=A[0]),
    dict(y=A[0], ldx=264), dict(out_dtype="e4m3", scale=A[6], y=A[0]),
    dict(out_dtype="e4m3", scale=A[5]), dict(out_dtype="e4m3", scale=A[6] + 1),
    dict(T=1 << 62), dict(ldx=1 << 62)], ids=str)
def test_norm_invalid(change):
    assert _norm(**change) == INVALID


def test_norm_sizes():
    assert _norm(H=1 << 31) == UNSUPPORTED
    assert _norm(T=0) == ar.AR_OK
    assert _norm(T=0, H=0) == INVALID


def _grad(**kw):
    a = dict(dy=A[0], dtotal=A[1], total=A[2], gamma=A[3], rstd=A[4], dx=A[5], dgamma=A[6],
             work=A[7], work_bytes=4 * 256 * 4, T=4, H=256, dtype="bf16")
    a.update(kw)
    return _code(ar.ar_rmsnorm_grad, **a)


@pytest.mark.parametrize("change", [
    dict(dy=None), dict(total=None), dict(rstd=None), dict(dx=None), dict(work=None),
    dict(dgamma=None), dict(work_bytes=4 * 256 * 4 - 1), dict(work=A[7] + 4), dict(H=0),
    dict(dtype="e4m3"), dict(dy=A[0] + 1), dict(dgamma=A[6] + 2), dict(rstd=A[4] + 1),
    dict(dx=A[0] + 2), dict(dx=A[3]), dict(dx=A[0], lddy=300), dict(work=A[0]), dict(work=A[5]),
    dict(dgamma=A[7] + 16), dict(dgamma=A[2]), dict(lddy=3), dict(lddtotal=3), dict(ldtotal=3),
    dict(lddx=255), dict(T=1 << 61)], ids=str)
def test_norm_grad_invalid(change):
    assert _grad(**change) == INVALID


def test_norm_grad_sizes():
    assert _grad(H=1 << 31) == UNSUPPORTED
    assert _grad(T=0, dgamma=None, work=None) == ar.AR_OK


def _route(**kw):
    a = dict(ids=A[0], T=16, K=8, E=64, offsets=A[1], row_of=A[2], src=A[3], ids_bytes=4)
    a.update(kw)
    return _code(ar.ar_moe_route, **a)


@pytest.mark.parametrize("change", [
    dict(ids=None), dict(offsets=None), dict(row_of=None), dict(K=0), dict(K=33), dict(E=0),
    dict(E=-1), dict(ids_bytes=2), dict(ids=A[0] + 2), dict(ids=A[0] + 4, ids_bytes=8),
    dict(offsets=A[1] + 1), dict(row_of=A[2] + 2), dict(src=A[3] + 1), dict(offsets=A[0]),
    dict(row_of=A[0]), dict(src=A[2] + 4), dict(offsets=A[2])], ids=str)
def test_route_invalid(change):
    assert _route(**change) == INVALID


def test_route_sizes():
    assert _route(E=1025) == UNSUPPORTED
    assert _route(T=1 << 28) == UNSUPPORTED
    assert _route(T=1 << 62) == UNSUPPORTED


def _dispatch(**kw):
    a = dict(x=A[0], xscale=A[1], row_of=A[2], rows=A[3], rscale=A[4], nrows=128, T=16, K=8,
             H=256, dtype="e4m3")
    a.update(kw)
    return _code(ar.ar_moe_dispatch, **a)


@pytest.mark.parametrize("change", [
    dict(x=None), dict(row_of=None), dict(rows=None), dict(xscale=None), dict(rscale=None),
    dict(K=0), dict(K=33), dict(H=0), dict(dtype=7), dict(dtype="bf16", x=A[0] + 1),
    dict(dtype="fp32", rows=A[3] + 2), dict(row_of=A[2] + 1), dict(rscale=A[4] + 1),
    dict(rows=A[0] + 16), dict(rows=A[0]), dict(rscale=A[1]), dict(rscale=A[3]), dict(ldx=255),
    dict(ldrows=128), dict(nrows=1 << 60)], ids=str)
def test_dispatch_invalid(change):
    assert _dispatch(**change) == INVALID


def _return(**kw):
    a = dict(rows=A[0], nrows=128, row_of=A[1], w=A[2], out=A[3], T=16, K=8, H=256, dtype="bf16")
    a.update(kw)
    return _code(ar.ar_moe_return, **a)


@pytest.mark.parametrize("change", [
    dict(rows=None), dict(row_of=None), dict(out=None), dict(K=0), dict(K=33), dict(H=0),
    dict(dtype="e4m3"), dict(rows=A[0] + 1), dict(w=A[2] + 2), dict(out=A[3] + 1),
    dict(row_of=A[1] + 2), dict(out=A[0]), dict(out=A[0] + 512), dict(out=A[2]), dict(out=A[1]),
    dict(ldrows=100), dict(ldout=100)], ids=str)
def test_return_invalid(change):
    assert _return(**change) == INVALID


def _return_grad(**kw):
    a = dict(dout=A[0], rows=A[1], nrows=128, row_of=A[2], w=A[3], drows=A[4], dw=A[5], T=16, K=8,
             H=256, dtype="bf16")
    a.update(kw)
    return _code(ar.ar_moe_return_grad, **a)


@pytest.mark.parametrize("change", [
    dict(dout=None), dict(rows=None), dict(row_of=None), dict(drows=None, dw=None), dict(K=0),
    dict(K=33), dict(H=0), dict(dtype="e4m3"), dict(dout=A[0] + 1), dict(rows=A[1] + 1),
    dict(drows=A[4] + 1), dict(w=A[3] + 1), dict(dw=A[5] + 1), dict(drows=A[1] + 512),
    dict(drows=A[1], ldrows=300), dict(drows=A[0]), dict(drows=A[3]), dict(dw=A[3]),
    dict(dw=A[4]), dict(dw=A[1]), dict(lddout=1), dict(ldrows=1), dict(lddrows=1)], ids=str)
def test_return_grad_invalid(change):
    assert _return_grad(**change) == INVALID


def test_row_mover_sizes():
    for call in (_dispatch, _return, _return_grad):
        assert call(T=1 << 28) == UNSUPPORTED
        assert call(H=1 << 31) == UNSUPPORTED
        assert call(T=0) == ar.AR_OK


def _matmul(**kw):
    a = dict(a=A[0], sa=A[1], b=A[2], sb=A[3], offsets=A[4], E=4, d=A[5], M=64, N=256, K=512,
             out_dtype="bf16", status=A[6])
    a.update(kw)
    return _code(ar.ar_matmul8, **a)


@pytest.mark.parametrize("change", [
    dict(a=None), dict(sa=None), dict(b=None), dict(sb=None), dict(d=None), dict(offsets=None),
    dict(N=0), dict(K=0), dict(E=0), dict(E=-3), dict(out_dtype="e4m3"), dict(lda=511),
    dict(ldb=500), dict(ldd=255), dict(d=A[5] + 1), dict(sa=A[1] + 2), dict(sb=A[3] + 1),
    dict(offsets=A[4] + 2), dict(status=A[6] + 1), dict(d=A[0]), dict(d=A[2] + 512), dict(d=A[1]),
    dict(d=A[3]), dict(d=A[4]), dict(status=A[5] + 4), dict(ldb=1 << 62)], ids=str)
def test_matmul8_invalid(change):
    assert _matmul(**change) == INVALID


def test_matmul8_sizes():
    for big in (dict(M=1 << 31), dict(N=1 << 31), dict(K=1 << 31), dict(E=1025)):
        assert _matmul(**big) == UNSUPPORTED
    assert _matmul(M=0) == ar.AR_OK
