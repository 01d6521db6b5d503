"""The host side of the layer operators, on the CPU: limits, and what the binding
makes of its arguments.  No call here launches anything."""
import os
import sys
import sysconfig

import pytest

import all_reduce_reduction_gb300 as ar
from all_reduce_reduction_gb300 import build as cuda_build

A = [0x10000000 * (i + 1) for i in range(10)]


@pytest.fixture(scope="module", autouse=True)
def built():
    cuda_build.build()


def _code(fn, *args, **kw):
    try:
        fn(*args, stream=0, **kw)
    except ar.ArError as e:
        return e.code
    return ar.AR_OK


@pytest.mark.parametrize("K", [1, 2, 3, 7, 8, 29, 32])
def test_pairs_are_taken_up_to_the_stated_limit(K):
    """T * K < 2^31; with the limit kept the calls go on to the missing pointer."""
    most = (2 ** 31 - 1) // K
    for T, code in ((most, ar.AR_ERR_INVALID), (most + 1, ar.AR_ERR_UNSUPPORTED)):
        assert _code(ar.ar_moe_route, None, T, K, 64, A[0], A[1]) == code
        assert _code(ar.ar_moe_dispatch, None, None, A[0], A[1], None, 8, T, K, 64, "bf16") == code
        assert _code(ar.ar_moe_return, None, 8, A[0], None, A[1], T, K, 64, "bf16") == code
        assert _code(ar.ar_moe_return_grad, None, A[0], 8, A[1], None, A[2], None, T, K, 64,
                     "bf16") == code


class _Recorder:
    """Stands in for the extension module; keeps what a call was given."""

    def __getattr__(self, name):
        def call(*args):
            self.args = args
            return ar.AR_OK
        return call


class _Ids:
    def __init__(self, size):
        self.size = size

    def data_ptr(self):
        return A[0]

    def element_size(self):
        return self.size


@pytest.mark.parametrize("ids,given,want", [
    (_Ids(8), {}, 8), (_Ids(4), {}, 4), (_Ids(2), {}, 2), (_Ids(8), dict(ids_bytes=4), 4),
    (A[0], {}, 4), (A[0], dict(ids_bytes=8), 8), (None, {}, 4)])
def test_route_takes_the_width_of_its_ids(monkeypatch, ids, given, want):
    """A tensor's own element size, 4 for an address, and always what the caller says."""
    calls = _Recorder()
    monkeypatch.setattr(ar, "_calls", calls)
    ar.ar_moe_route(ids, 16, 8, 64, A[1], A[2], stream=0, **given)
    assert calls.args[0] is ids and calls.args[1] == want


def test_route_refuses_ids_of_another_width():
    assert _code(ar.ar_moe_route, _Ids(2), 16, 8, 64, A[1], A[2]) == ar.AR_ERR_INVALID


def test_the_module_names_its_interpreter():
    """One built for another interpreter is neither fresh nor loaded."""
    suffix = sysconfig.get_config_var("EXT_SUFFIX")
    assert cuda_build.NATIVE.endswith("_native" + suffix) and suffix != ".so"
    assert ar._layer_calls().__file__ == cuda_build.NATIVE


@pytest.fixture
def no_headers(monkeypatch, tmp_path):
    """A machine without Python's headers, where no module was built."""
    monkeypatch.setattr(sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    monkeypatch.setattr(cuda_build, "NATIVE", str(tmp_path / "_native.so"))
    monkeypatch.setattr(ar, "_calls", None)
    monkeypatch.setattr(ar, "_NATIVE_PATH", str(tmp_path / "_native.so"), raising=False)
    monkeypatch.delitem(sys.modules, ar.__name__ + "._native", raising=False)


def test_the_library_builds_without_python_headers(no_headers, capfd):
    before = os.path.getmtime(cuda_build.LIB)
    assert cuda_build.build() == cuda_build.LIB
    assert not os.path.exists(cuda_build.NATIVE) and "Python.h" in capfd.readouterr().err
    assert os.path.getmtime(cuda_build.LIB) == before        # which was up to date


def test_the_calls_without_the_module(no_headers):
    """Through ctypes: the same answers and refusals."""
    assert _code(ar.ar_rmsnorm, A[0], None, None, 1e-6, None, A[1], None, None, 0, 64,
                 "bf16") == ar.AR_OK
    assert _code(ar.ar_rmsnorm, None, None, None, 1e-6, None, A[1], None, None, 1, 64,
                 "bf16") == ar.AR_ERR_INVALID
    assert _code(ar.ar_moe_route, _Ids(2), 16, 8, 64, A[1], A[2]) == ar.AR_ERR_INVALID
    assert _code(ar.ar_matmul8, A[0], A[1], A[2], A[3], None, 1, A[4], 0, 64, 64,
                 "bf16") == ar.AR_OK
    for bad in (dict(T=-1), dict(T=1.5), dict(H=2 ** 64), dict(dtype=2 ** 31), dict(x="text"),
                dict(stream="x"), dict(eps="x")):
        a = dict(x=A[0], res=None, gamma=None, eps=1e-6, total=None, y=A[1], scale=None, rstd=None,
                 T=0, H=64, dtype="bf16", stream=0) | bad
        with pytest.raises((TypeError, ValueError, OverflowError, AttributeError)):
            ar.ar_rmsnorm(**a)
    with pytest.raises(TypeError):
        ar._layer_calls().ar_moe_route(0, 4)
    assert "_native" not in [m.split(".")[-1] for m in sys.modules if m.startswith(ar.__name__)]
