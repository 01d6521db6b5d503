"""The extension module that converts the layer operators' arguments, on the CPU:
calls of zero rows return before any CUDA call."""
import sys

import pytest

import all_reduce_reduction_gb300 as ar
from all_reduce_reduction_gb300 import build as cuda_build


@pytest.fixture(scope="module")
def calls():
    cuda_build.build()
    return ar._layer_calls()


class Tensor:
    def __init__(self, ptr):
        self.ptr = ptr

    def data_ptr(self):
        return self.ptr


class Stream:
    cuda_stream = 0x1234


def _norm(x=0x1000, T=0, H=64, eps=1e-6, dtype=0, stream=0):
    return (x, 0, None, 0, None, eps, None, 0, 0x2000, 0, None, None, T, H, dtype, dtype, stream)


def test_pointers_and_streams(calls):
    for x in (0x1000, Tensor(0x1000), Tensor(2 ** 63 + 16), None):
        assert calls.ar_rmsnorm(*_norm(x=x)) == ar.AR_OK
    for s in (0, 0xABC, Stream()):
        assert calls.ar_rmsnorm(*_norm(stream=s)) == ar.AR_OK
    assert calls.ar_rmsnorm(*_norm(x=None, T=1)) == ar.AR_ERR_INVALID
    assert calls.ar_rmsnorm(*_norm(x=Tensor(0x1001), T=1)) == ar.AR_ERR_INVALID


@pytest.mark.parametrize("change", [
    dict(x="text"), dict(x=1.5), dict(x=Tensor("text")), dict(T=-1), dict(T=1.5), dict(H=2 ** 64),
    dict(dtype=2 ** 31), dict(dtype="int8"), dict(eps="x"), dict(stream="x")], ids=str)
def test_arguments_that_do_not_convert(calls, change):
    with pytest.raises((TypeError, ValueError, OverflowError, AttributeError)):
        calls.ar_rmsnorm(*_norm(**change))


def test_argument_counts(calls):
    for name, n in [("ar_rmsnorm", 17), ("ar_rmsnorm_grad", 17), ("ar_moe_route", 9),
                    ("ar_moe_dispatch", 13), ("ar_moe_return", 12), ("ar_moe_return_grad", 15),
                    ("ar_matmul8", 16)]:
        assert len(ar.SIGNATURES[name][0]) == n
        for k in (0, n - 1, n + 1):
            with pytest.raises(TypeError):
                getattr(calls, name)(*([0] * k))


def test_no_reference_is_lost(calls):
    t, s, n = Tensor(0x1000), Stream(), 10 ** 6 + 7
    before = [sys.getrefcount(o) for o in (t, s, n)]
    for _ in range(100):
        calls.ar_rmsnorm(*_norm(x=t, H=n, stream=s))
    assert [sys.getrefcount(o) for o in (t, s, n)] == before
