"""GB300-native sum all-reduce over R virtual ranks held in one GPU's HBM.

This module is a thin ctypes binding of the C ABI declared in
``include/ar.h`` (library ``libar_gb300.so``, built in-tree by
``all_reduce_reduction_gb300.build``), but for the layer operators, which call
it through a small extension module (through ctypes too where that was not
built).  Every function has the name of the C entry point it calls and only
marshals arguments: device buffers may be given as integers (device addresses)
or as objects with ``data_ptr()`` (torch CUDA tensors); a stream as an integer
``cudaStream_t``, an object with ``cuda_stream`` (``torch.cuda.Stream``), or
``None`` for torch's current stream.  All work runs in the library's CUDA
kernels; there is no CPU path.
If the library is missing, the first call raises ``RuntimeError``.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import sysconfig
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libar_gb300.so")

# enum ar_dtype / ar_algo / ar_proto / ar_status_code (include/ar.h)
AR_BF16, AR_FP16, AR_FP32 = 0, 1, 2
AR_ONE_SHOT, AR_TWO_SHOT, AR_ALGO_AUTO = 0, 1, 2
AR_LL, AR_HB, AR_PROTO_AUTO = 0, 1, 2
AR_OK = 0
AR_ERR_INVALID = 1
AR_ERR_UNSUPPORTED = 2
AR_ERR_CUDA = 3
AR_ERR_NOMEM = 4
AR_ERR_TIMEOUT = 5
AR_ERR_FLAG_MISMATCH = 6
AR_LL_AUTO, AR_LL_GLOBAL, AR_LL_CLUSTER = 0, 1, 2
AR_HB_STAGING_AUTO, AR_HB_STAGING_TMA, AR_HB_STAGING_DIRECT = 0, 1, 2
AR_MAX_RANKS = 32
AR_LL_MAX_BYTES = 64 << 20
AR_E4M3 = 8                     # enum ar_dtype8
AR_SCALE_BLOCK = 128
AR_MOE_MAX_EXPERTS = 1024
AR_MOE_MAX_CHOICES = 32
AR_NORM_GRAD_ROWS = 512
AR_CACHE_MAX_DIM = 256
AR_CACHE_MAX_HEADS = 1024
AR_CACHE_WORK_ROWS = 16384
AR_MOE_LAYER_TOKENS = 64
AR_MOE_LAYER_PAIRS = 512

DTYPES = {"bf16": AR_BF16, "fp16": AR_FP16, "fp32": AR_FP32}
DTYPES8 = {**DTYPES, "e4m3": AR_E4M3}
ALGOS = {"one_shot": AR_ONE_SHOT, "two_shot": AR_TWO_SHOT, "auto": AR_ALGO_AUTO}
PROTOS = {"ll": AR_LL, "hb": AR_HB, "auto": AR_PROTO_AUTO}


class ArError(RuntimeError):
    """A nonzero ar_status_code returned by the library."""

    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__("%s: %s" % (where, ar_strerror(code)))


class ar_info(ctypes.Structure):
    _fields_ = [
        ("R", ctypes.c_int),
        ("dtype", ctypes.c_int),
        ("N", ctypes.c_size_t),
        ("elem_size", ctypes.c_size_t),
        ("ll_capable", ctypes.c_int),
        ("ll_packets_per_rank", ctypes.c_size_t),
        ("scratch_bytes", ctypes.c_size_t),
        ("num_sms", ctypes.c_int),
        ("ll_ctas_per_rank_max", ctypes.c_int),
        ("tma_tile_bytes", ctypes.c_int),
        ("tma_stages", ctypes.c_int),
        ("timeout_ns", ctypes.c_uint64),
        ("ll_transport", ctypes.c_int),
        ("ll_cluster_ok", ctypes.c_int),
        ("ll_cluster_units", ctypes.c_int),
        ("ll_cluster_max", ctypes.c_int),
        ("pdl", ctypes.c_int),
        ("ll_staged_ctas_max", ctypes.c_int),
        ("hb_staging", ctypes.c_int),
    ]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


AR_OP_COPY, AR_OP_REDUCE = 0, 1
AR_BUF_IN, AR_BUF_OUT = 0, 1


class ar_op(ctypes.Structure):
    _fields_ = [
        ("kind", ctypes.c_int),
        ("rank", ctypes.c_int),
        ("dst_buf", ctypes.c_int),
        ("dst_rank", ctypes.c_int),
        ("src_buf", ctypes.c_int),
        ("nsrc", ctypes.c_int),
        ("src_rank", ctypes.c_int * AR_MAX_RANKS),
        ("chunk_begin", ctypes.c_int),
        ("chunk_end", ctypes.c_int),
    ]


_lock = threading.Lock()
_lib = None

# exported entry points: name -> (argtypes, restype)
_VP, _SZ, _I, _U32, _U64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_uint32, ctypes.c_uint64
_VPP = ctypes.POINTER(ctypes.c_void_p)
SIGNATURES = {
    "ar_create": ([_I, _SZ, _I, ctypes.POINTER(_VP)], _I),
    "ar_destroy": ([_VP], _I),
    "ar_allreduce": ([_VP, _VPP, _VPP, _I, _I, _VP], _I),
    "ar_allreduce_n": ([_VP, _VPP, _VPP, _SZ, _I, _I, _VP], _I),
    "ar_allreduce_host": ([_VP, _VPP, _VPP, _SZ, _I, _I, _VP], _I),
    "ar_tune": ([_VP, _VP], _I),
    "ar_combine": ([_VP, _VPP, _VP, _VP, _SZ, _SZ, _VP], _I),
    "ar_get_tuning": ([_VP, _SZ, ctypes.POINTER(_I), ctypes.POINTER(_I),
                       ctypes.POINTER(ctypes.c_float)], _I),
    "ar_reduce_scatter": ([_VP, _VPP, _VPP, _VP], _I),
    "ar_all_gather": ([_VP, _VPP, _VP], _I),
    "ar_ll_pack": ([_VP, _VP, _VP, _SZ, _U32, _VP], _I),
    "ar_ll_unpack": ([_VP, _VP, _VP, _SZ, _U32, _VP], _I),
    "ar_status": ([_VP, _VP], _I),
    "ar_set_timeout": ([_VP, _U64], _I),
    "ar_debug_drop_rank": ([_VP, _I], _I),
    "ar_set_ll_transport": ([_VP, _I], _I),
    "ar_set_hb_staging": ([_VP, _I], _I),
    "ar_get_hb_staging": ([_VP, _SZ, ctypes.POINTER(_I)], _I),
    "ar_set_grid_divisor": ([_VP, _I], _I),
    "ar_get_grid_divisor": ([_VP, _SZ, _I, _I, ctypes.POINTER(_I)], _I),
    "ar_set_pdl": ([_VP, _I], _I),
    "ar_round": ([_I, _VP, _VP, _SZ, _VP], _I),
    "ar_get_info": ([_VP, ctypes.POINTER(ar_info)], _I),
    "ar_strerror": ([_I], ctypes.c_char_p),
    "ar_allreduce_ll_static": ([_I, _SZ, _I, _VPP, _VPP, _VP], _I),
    "ar_plan_compile": ([_VP, ctypes.POINTER(ar_op), _I, _I, _I, ctypes.POINTER(_VP)], _I),
    "ar_plan_builtin": ([_VP, _I, _I, _I, ctypes.POINTER(_VP)], _I),
    "ar_plan_execute": ([_VP, _VPP, _VPP, _VP], _I),
    "ar_plan_stats": ([_VP, ctypes.POINTER(_I), ctypes.POINTER(_I), ctypes.POINTER(_I)], _I),
    "ar_plan_destroy": ([_VP], _I),
    "ar_rmsnorm": ([_VP, _SZ, _VP, _SZ, _VP, ctypes.c_float, _VP, _SZ, _VP, _SZ, _VP, _VP, _SZ,
                    _SZ, _I, _I, _VP], _I),
    "ar_rmsnorm_grad": ([_VP, _SZ, _VP, _SZ, _VP, _SZ, _VP, _VP, _VP, _SZ, _VP, _VP, _SZ, _SZ,
                         _SZ, _I, _VP], _I),
    "ar_moe_route": ([_VP, _I, _SZ, _I, _I, _VP, _VP, _VP, _VP], _I),
    "ar_moe_dispatch": ([_VP, _SZ, _VP, _VP, _VP, _SZ, _VP, _SZ, _SZ, _I, _SZ, _I, _VP], _I),
    "ar_moe_return": ([_VP, _SZ, _SZ, _VP, _VP, _VP, _SZ, _SZ, _I, _SZ, _I, _VP], _I),
    "ar_moe_return_grad": ([_VP, _SZ, _VP, _SZ, _SZ, _VP, _VP, _VP, _SZ, _VP, _SZ, _I, _SZ, _I,
                            _VP], _I),
    "ar_matmul8": ([_VP, _SZ, _VP, _VP, _SZ, _VP, _VP, _I, _VP, _SZ, _SZ, _SZ, _SZ, _I, _VP,
                    _VP], _I),
    "ar_cache_write": ([_VP, _SZ, _VP, _SZ, _VP, _VP, _SZ, _VP, _VP, _SZ, _I, _VP, _SZ, _SZ, _VP,
                        _VP, _SZ, _SZ, _I, _I, _I, _I, _VP], _I),
    "ar_cache_read": ([_VP, _VP, _SZ, _VP, _VP, _SZ, _I, _VP, _SZ, _SZ, _VP, _VP, _VP, _SZ, _VP,
                       _SZ, _SZ, _SZ, _I, _I, _I, _I, _VP], _I),
    "ar_cache_attention": ([_VP, _SZ, _VP, _VP, _SZ, _VP, _VP, _SZ, _I, _VP, _SZ, _SZ, _VP,
                            ctypes.c_float, _SZ, _VP, _SZ, _VP, _VP, _SZ, _SZ, _I, _I, _I, _I, _I,
                            _VP], _I),
    "ar_moe_layer": ([_VP, _SZ, _VP, _I, _VP, _VP, _SZ, _VP, _VP, _SZ, _VP, _VP, _SZ, _VP, _SZ,
                      _SZ, _I, _I, _SZ, _SZ, _I, _VP], _I),
}


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the CUDA library (no GPU call is made).  Raises if it is absent."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    with _lock:
        if _lib is not None and path == LIB_PATH:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(
                "libar_gb300.so is not built (expected at %s); run "
                "`python -c 'import __graft_entry__ as g; g.build()'`" % path)
        lib = ctypes.CDLL(path)
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = args, res
        if path == LIB_PATH:
            _lib = lib
        return lib


def _ptr(x) -> int:
    if x is None:
        return 0
    if isinstance(x, int):
        return x
    return x.data_ptr()


_raw_stream = None            # torch's (raw stream of a device, current device)


def _current_stream() -> int:
    """The caller's current CUDA stream as an integer.  torch's raw lookup
    answers in a tenth of the time of building a Stream object, which was most
    of a small call's host cost (3 us); it is an internal name of torch, so the
    public way stays where it is missing."""
    global _raw_stream
    if _raw_stream is None:
        import torch
        names = ("_cuda_getCurrentRawStream", "_cuda_getDevice")
        if not torch.cuda.is_initialized() or not all(hasattr(torch._C, n) for n in names):
            return int(torch.cuda.current_stream().cuda_stream)
        _raw_stream = tuple(getattr(torch._C, n) for n in names)
    return _raw_stream[0](_raw_stream[1]())


def _stream(s) -> int:
    if s is None:
        return _current_stream()
    if isinstance(s, int):
        return s
    return int(s.cuda_stream)


def _ptr_array(bufs):
    """Host array of device pointers, always AR_MAX_RANKS long: entries past
    the given buffers are NULL, so passing fewer buffers than the handle's
    ranks is rejected by the library (AR_ERR_INVALID) instead of reading past
    the end of the array."""
    if len(bufs) > AR_MAX_RANKS:
        raise ValueError("at most %d buffers" % AR_MAX_RANKS)
    arr = (ctypes.c_void_p * AR_MAX_RANKS)()
    for i, b in enumerate(bufs):
        arr[i] = _ptr(b)
    return arr


def _check(code: int, where: str) -> None:
    if code != AR_OK:
        raise ArError(code, where)


def ar_strerror(code: int) -> str:
    return load_library().ar_strerror(code).decode()


def ar_create(R: int, N: int, dtype) -> int:
    """Create a handle for R ranks of N elements; returns it as an integer."""
    dt = DTYPES[dtype] if isinstance(dtype, str) else dtype
    h = ctypes.c_void_p()
    _check(load_library().ar_create(R, N, dt, ctypes.byref(h)), "ar_create")
    return h.value


def ar_destroy(h: int) -> None:
    _check(load_library().ar_destroy(h), "ar_destroy")


def ar_allreduce(h: int, ins, outs, algo=AR_ONE_SHOT, proto=AR_HB, stream=None) -> None:
    algo = ALGOS[algo] if isinstance(algo, str) else algo
    proto = PROTOS[proto] if isinstance(proto, str) else proto
    _check(load_library().ar_allreduce(h, _ptr_array(ins), _ptr_array(outs), algo, proto,
                                       _stream(stream)), "ar_allreduce")


def ar_allreduce_n(h: int, ins, outs, n: int, algo=AR_ALGO_AUTO, proto=AR_PROTO_AUTO,
                   stream=None) -> None:
    algo = ALGOS[algo] if isinstance(algo, str) else algo
    proto = PROTOS[proto] if isinstance(proto, str) else proto
    _check(load_library().ar_allreduce_n(h, _ptr_array(ins), _ptr_array(outs), n, algo, proto,
                                         _stream(stream)), "ar_allreduce_n")


def ar_allreduce_host(h: int, ins, outs, n: int, algo=AR_ALGO_AUTO, proto=AR_PROTO_AUTO,
                      stream=None) -> None:
    algo = ALGOS[algo] if isinstance(algo, str) else algo
    proto = PROTOS[proto] if isinstance(proto, str) else proto
    _check(load_library().ar_allreduce_host(h, _ptr_array(ins), _ptr_array(outs), n, algo, proto,
                                            _stream(stream)), "ar_allreduce_host")


def ar_combine(h: int, ys, w, out, T: int, H: int, stream=None) -> None:
    _check(load_library().ar_combine(h, _ptr_array(ys), _ptr(w), _ptr(out), T, H,
                                      _stream(stream)), "ar_combine")


def ar_tune(h: int, stream=None) -> None:
    _check(load_library().ar_tune(h, _stream(stream)), "ar_tune")


def ar_get_tuning(h: int, nbytes: int):
    """(algo, proto, [µs one-shot LL, one-shot HB, two-shot LL, two-shot HB])."""
    a, p = ctypes.c_int(), ctypes.c_int()
    us = (ctypes.c_float * 4)()
    _check(load_library().ar_get_tuning(h, nbytes, ctypes.byref(a), ctypes.byref(p), us),
           "ar_get_tuning")
    return a.value, p.value, list(us)


def ar_reduce_scatter(h: int, ins, outs, stream=None) -> None:
    _check(load_library().ar_reduce_scatter(h, _ptr_array(ins), _ptr_array(outs), _stream(stream)),
           "ar_reduce_scatter")


def ar_all_gather(h: int, outs, stream=None) -> None:
    _check(load_library().ar_all_gather(h, _ptr_array(outs), _stream(stream)), "ar_all_gather")


def ar_ll_pack(h: int, src, pkts, n: int, flag: int, stream=None) -> None:
    _check(load_library().ar_ll_pack(h, _ptr(src), _ptr(pkts), n, flag & 0xFFFFFFFF,
                                     _stream(stream)), "ar_ll_pack")


def ar_ll_unpack(h: int, pkts, dst, n: int, flag: int, stream=None) -> None:
    _check(load_library().ar_ll_unpack(h, _ptr(pkts), _ptr(dst), n, flag & 0xFFFFFFFF,
                                       _stream(stream)), "ar_ll_unpack")


def ar_status(h: int, stream=None) -> int:
    """Wait for the stream; return (and clear) the handle's device status."""
    return load_library().ar_status(h, _stream(stream))


def ar_set_timeout(h: int, ns: int) -> None:
    _check(load_library().ar_set_timeout(h, ns), "ar_set_timeout")


def ar_set_pdl(h: int, enable: int) -> None:
    _check(load_library().ar_set_pdl(h, enable), "ar_set_pdl")


def ar_set_ll_transport(h: int, transport: int) -> None:
    _check(load_library().ar_set_ll_transport(h, transport), "ar_set_ll_transport")


def ar_set_hb_staging(h: int, staging: int) -> None:
    _check(load_library().ar_set_hb_staging(h, staging), "ar_set_hb_staging")


def ar_get_hb_staging(h: int, nbytes: int) -> int:
    """AR_HB_STAGING_TMA or AR_HB_STAGING_DIRECT: what a two-shot HB call of
    `nbytes` per rank (16-byte-aligned buffers) would use now."""
    out = ctypes.c_int(0)
    _check(load_library().ar_get_hb_staging(h, nbytes, ctypes.byref(out)), "ar_get_hb_staging")
    return out.value


def ar_set_grid_divisor(h: int, divisor: int) -> None:
    """Force the CTA-cap divisor of later calls (1, 2, 4, 8; 0 = tuned)."""
    _check(load_library().ar_set_grid_divisor(h, divisor), "ar_set_grid_divisor")


def ar_get_grid_divisor(h: int, nbytes: int, algo, proto) -> int:
    """The CTA-cap divisor a call of `nbytes` per rank with this algo and
    proto would use now."""
    algo = ALGOS[algo] if isinstance(algo, str) else algo
    proto = PROTOS[proto] if isinstance(proto, str) else proto
    out = ctypes.c_int(0)
    _check(load_library().ar_get_grid_divisor(h, nbytes, algo, proto, ctypes.byref(out)),
           "ar_get_grid_divisor")
    return out.value


def ar_debug_drop_rank(h: int, rank: int) -> None:
    _check(load_library().ar_debug_drop_rank(h, rank), "ar_debug_drop_rank")


def ar_round(dtype, src, dst, n: int, stream=None) -> None:
    dt = DTYPES[dtype] if isinstance(dtype, str) else dtype
    _check(load_library().ar_round(dt, _ptr(src), _ptr(dst), n, _stream(stream)), "ar_round")


def ar_get_info(h: int) -> dict:
    info = ar_info()
    _check(load_library().ar_get_info(h, ctypes.byref(info)), "ar_get_info")
    return info.as_dict()


def ar_allreduce_ll_static(R: int, N: int, dtype, ins, outs, stream=None) -> None:
    """One-shot LL all-reduce with no handle and no allocation, for callers
    that may not allocate device memory where they run it: an engine whose
    own pool holds nearly all of the GPU's memory, or a latency-critical
    hook that cannot pay for cudaMalloc's device-wide synchronisation.  The
    packet scratch is a static array inside the library (at most
    AR_NOALLOC_SCRATCH_BYTES of packets, else AR_ERR_UNSUPPORTED); the first
    call on a device sets it up and waits for that to finish; calls that
    overlap on the GPU race on the shared array."""
    dt = DTYPES[dtype] if isinstance(dtype, str) else dtype
    _check(load_library().ar_allreduce_ll_static(R, N, dt, _ptr_array(ins), _ptr_array(outs),
                                                 _stream(stream)), "ar_allreduce_ll_static")


AR_NOALLOC_SCRATCH_BYTES = 8 << 20


def make_op(kind, rank, dst, srcs, chunk_begin, chunk_end) -> ar_op:
    """One plan step.  dst = (buf, rank); srcs = [(buf, rank), ...] (all of
    one buffer kind)."""
    o = ar_op()
    o.kind = kind
    o.rank = rank
    o.dst_buf, o.dst_rank = dst
    o.src_buf = srcs[0][0]
    o.nsrc = len(srcs)
    for i, (b, r) in enumerate(srcs):
        if b != o.src_buf:
            raise ValueError("the sources of one step share a buffer kind")
        o.src_rank[i] = r
    o.chunk_begin, o.chunk_end = chunk_begin, chunk_end
    return o


def ar_plan_compile(h: int, ops, nchunks: int, ctas_per_rank: int = 1) -> int:
    arr = (ar_op * len(ops))(*ops)
    p = ctypes.c_void_p()
    _check(load_library().ar_plan_compile(h, arr, len(ops), nchunks, ctas_per_rank,
                                          ctypes.byref(p)), "ar_plan_compile")
    return p.value


def ar_plan_builtin(h: int, algo, chunks_per_rank: int = 0, ctas_per_rank: int = 0) -> int:
    algo = ALGOS[algo] if isinstance(algo, str) else algo
    p = ctypes.c_void_p()
    _check(load_library().ar_plan_builtin(h, algo, chunks_per_rank, ctas_per_rank,
                                          ctypes.byref(p)), "ar_plan_builtin")
    return p.value


def ar_plan_execute(p: int, ins, outs, stream=None) -> None:
    _check(load_library().ar_plan_execute(p, _ptr_array(ins), _ptr_array(outs), _stream(stream)),
           "ar_plan_execute")


def ar_plan_stats(p: int):
    t, w, s = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    _check(load_library().ar_plan_stats(p, ctypes.byref(t), ctypes.byref(w), ctypes.byref(s)),
           "ar_plan_stats")
    return t.value, w.value, s.value


def ar_plan_destroy(p: int) -> None:
    _check(load_library().ar_plan_destroy(p), "ar_plan_destroy")


# The layer operators.  A decode step makes several of these calls per layer, and
# the host's share of a small one is most of its time, so they reach the library
# through an extension module that converts their arguments itself (one row of
# ar_rmsnorm: 3.1 us of conversion with ctypes, 1 with it).

_calls = None                  # the extension module _native, or what stands in for it
# the running interpreter's own
_NATIVE_PATH = os.path.join(HERE, "_native" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))


class _CtypesCalls:
    """The extension module's calls through ctypes, for an interpreter without it
    (no Python.h when the library was built).  One row of ar_rmsnorm takes 8.1 us a
    call so, 3.9 with the module."""

    def __getattr__(self, name):
        fn, kinds = getattr(load_library(), name), SIGNATURES[name][0]
        whole = {_SZ: (0, 1 << 64), _I: (-1 << 31, 1 << 31)}

        def call(*args):
            if len(args) != len(kinds):
                raise TypeError("%d arguments expected, %d given" % (len(kinds), len(args)))
            given = []
            for a, kind in zip(args[:-1], kinds):
                if kind in whole and not whole[kind][0] <= a < whole[kind][1]:
                    raise OverflowError("argument does not fit the C type")
                given.append(_ptr(a) if kind is _VP else a)
            try:
                return fn(*given, _stream(args[-1]))
            except ctypes.ArgumentError as e:
                raise TypeError(str(e)) from None
        setattr(self, name, call)
        return call


def _layer_calls():
    """The extension module, loaded with the library."""
    global _calls
    load_library()
    if _calls is None:
        if os.path.exists(_NATIVE_PATH):
            name = __name__ + "._native"
            spec = importlib.util.spec_from_file_location(name, _NATIVE_PATH)
            calls = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(calls)
            _calls = calls
        else:
            _calls = _CtypesCalls()
    return _calls


def ar_rmsnorm(x, res, gamma, eps: float, total, y, scale, rstd, T: int, H: int, dtype,
               out_dtype=None, ldx: int = 0, ldres: int = 0, ldsum: int = 0, ldy: int = 0,
               stream=None) -> None:
    """Residual addition and root-mean-square norm of T rows of H elements:
    ``total = x + res``, ``y = norm(x + res) * gamma`` in ``out_dtype`` (default
    ``dtype``; ``"e4m3"`` with one ``scale`` per 128 elements).  ``res``,
    ``gamma``, ``total``, ``scale`` and ``rstd`` may be None."""
    dt = DTYPES8.get(dtype, dtype)
    calls = _calls or _layer_calls()
    rc = calls.ar_rmsnorm(x, ldx, res, ldres, gamma, eps, total, ldsum, y, ldy, scale, rstd, T, H,
                          dt, dt if out_dtype is None else DTYPES8.get(out_dtype, out_dtype),
                          stream)
    if rc:
        raise ArError(rc, "ar_rmsnorm")


def ar_rmsnorm_grad(dy, dtotal, total, gamma, rstd, dx, dgamma, work, work_bytes: int, T: int,
                    H: int, dtype, lddy: int = 0, lddtotal: int = 0, ldtotal: int = 0,
                    lddx: int = 0, stream=None) -> None:
    """Gradient of ar_rmsnorm: ``dx`` (of x and of the residual alike) and the
    binary32 ``dgamma``, joined in ``work`` (min(T, AR_NORM_GRAD_ROWS) * H floats)."""
    calls = _calls or _layer_calls()
    rc = calls.ar_rmsnorm_grad(dy, lddy, dtotal, lddtotal, total, ldtotal, gamma, rstd, dx, lddx,
                               dgamma, work, work_bytes, T, H, DTYPES8.get(dtype, dtype), stream)
    if rc:
        raise ArError(rc, "ar_rmsnorm_grad")


def ar_moe_route(ids, T: int, K: int, E: int, offsets, row_of, src=None, ids_bytes=None,
                 stream=None) -> None:
    """Stable order of the T * K (token, choice) pairs by expert; ids outside
    [0, E) get no row.  ``ids_bytes`` (4 or 8) is a tensor's own element size
    unless given, and 4 for an address."""
    if ids_bytes is None:
        ids_bytes = ids.element_size() if hasattr(ids, "element_size") else 4
    calls = _calls or _layer_calls()
    rc = calls.ar_moe_route(ids, ids_bytes, T, K, E, offsets, row_of, src, stream)
    if rc:
        raise ArError(rc, "ar_moe_route")


def ar_moe_dispatch(x, xscale, row_of, rows, rscale, nrows: int, T: int, K: int, H: int, dtype,
                    ldx: int = 0, ldrows: int = 0, stream=None) -> None:
    """The tokens' rows (and their scales) in the experts' order."""
    calls = _calls or _layer_calls()
    rc = calls.ar_moe_dispatch(x, ldx, xscale, row_of, rows, ldrows, rscale, nrows, T, K, H,
                               DTYPES8.get(dtype, dtype), stream)
    if rc:
        raise ArError(rc, "ar_moe_dispatch")


def ar_moe_return(rows, nrows: int, row_of, w, out, T: int, K: int, H: int, dtype,
                  ldrows: int = 0, ldout: int = 0, stream=None) -> None:
    """The experts' rows back at their tokens, weighted (``w`` None: ones)."""
    calls = _calls or _layer_calls()
    rc = calls.ar_moe_return(rows, ldrows, nrows, row_of, w, out, ldout, T, K, H,
                             DTYPES8.get(dtype, dtype), stream)
    if rc:
        raise ArError(rc, "ar_moe_return")


def ar_moe_return_grad(dout, rows, nrows: int, row_of, w, drows, dw, T: int, K: int, H: int,
                       dtype, lddout: int = 0, ldrows: int = 0, lddrows: int = 0,
                       stream=None) -> None:
    """Gradient of ar_moe_return: of the rows and of the weights (either None)."""
    calls = _calls or _layer_calls()
    rc = calls.ar_moe_return_grad(dout, lddout, rows, ldrows, nrows, row_of, w, drows, lddrows, dw,
                                  T, K, H, DTYPES8.get(dtype, dtype), stream)
    if rc:
        raise ArError(rc, "ar_moe_return_grad")


def ar_matmul8(a, sa, b, sb, offsets, E: int, d, M: int, N: int, K: int, out_dtype,
               lda: int = 0, ldb: int = 0, ldd: int = 0, status=None, stream=None) -> None:
    """Product of E4M3 rows with E4M3 weights and their scales per block of
    128, for one matrix (``offsets`` None) or grouped by expert.  ``status``: an
    int32 word on the device, 0 before; a product whose wait ran out puts
    AR_ERR_TIMEOUT there and leaves ``d`` unfinished, which nothing else tells."""
    calls = _calls or _layer_calls()
    rc = calls.ar_matmul8(a, lda, sa, b, ldb, sb, offsets, E, d, ldd, M, N, K,
                          DTYPES8.get(out_dtype, out_dtype), status, stream)
    if rc:
        raise ArError(rc, "ar_matmul8")


def ar_cache_write(k, v, kcache, vcache, kscale, vscale, pages: int, page: int, table, width: int,
                   lens, offsets, T: int, B: int, heads: int, D: int, dtype, cache_dtype=None,
                   ldk: int = 0, ldv: int = 0, ldpage: int = 0, ldtable: int = 0,
                   stream=None) -> None:
    """New rows of keys and values into the pages of their sequences, in
    ``cache_dtype`` (default ``dtype``; ``"e4m3"`` with a scale for each row and
    head).  ``offsets`` None: one row a sequence."""
    dt = DTYPES8.get(dtype, dtype)
    calls = _calls or _layer_calls()
    rc = calls.ar_cache_write(k, ldk, v, ldv, kcache, vcache, ldpage, kscale, vscale, pages, page,
                              table, ldtable, width, lens, offsets, T, B, heads, D, dt,
                              dt if cache_dtype is None else DTYPES8.get(cache_dtype, cache_dtype),
                              stream)
    if rc:
        raise ArError(rc, "ar_cache_write")


def ar_cache_read(kcache, vcache, kscale, vscale, pages: int, page: int, table, width: int, lens,
                  offsets, k, v, T: int, B: int, heads: int, D: int, dtype, cache_dtype=None,
                  ldpage: int = 0, ldtable: int = 0, ldk: int = 0, ldv: int = 0,
                  stream=None) -> None:
    """The rows that ar_cache_write would put there, back in ``dtype``."""
    dt = DTYPES8.get(dtype, dtype)
    calls = _calls or _layer_calls()
    rc = calls.ar_cache_read(kcache, vcache, ldpage, kscale, vscale, pages, page, table, ldtable,
                             width, lens, offsets, k, ldk, v, ldv, T, B, heads, D, dt,
                             dt if cache_dtype is None else DTYPES8.get(cache_dtype, cache_dtype),
                             stream)
    if rc:
        raise ArError(rc, "ar_cache_read")


def ar_cache_attention(q, kcache, vcache, kscale, vscale, pages: int, page: int, table, width: int,
                       lens, scale: float, out, lse, work, work_bytes: int, B: int, heads: int,
                       kv_heads: int, D: int, dtype, cache_dtype=None, window: int = 0,
                       ldq: int = 0, ldpage: int = 0, ldtable: int = 0, ldout: int = 0,
                       stream=None) -> None:
    """Attention of one new token a sequence over its cache (the last ``window``
    positions of it, 0: all).  ``lse`` may be None; ``work``: AR_CACHE_WORK_ROWS *
    (D + 2) floats."""
    dt = DTYPES8.get(dtype, dtype)
    calls = _calls or _layer_calls()
    rc = calls.ar_cache_attention(q, ldq, kcache, vcache, ldpage, kscale, vscale, pages, page,
                                  table, ldtable, width, lens, scale, window, out, ldout, lse,
                                  work, work_bytes, B, heads, kv_heads, D, dt,
                                  dt if cache_dtype is None
                                  else DTYPES8.get(cache_dtype, cache_dtype), stream)
    if rc:
        raise ArError(rc, "ar_cache_attention")


def ar_moe_layer(x, ids, w, up, up_scale, down, down_scale, out, work, work_bytes: int, T: int,
                 K: int, E: int, H: int, F: int, dtype, ldx: int = 0, ldup: int = 0,
                 lddown: int = 0, ldout: int = 0, ids_bytes=None, stream=None) -> None:
    """A mixture-of-experts layer for a few tokens (T * K <= AR_MOE_LAYER_PAIRS): gated
    first product, second product and the weighted sum over a token's choices.
    ``ids_bytes`` as for ar_moe_route; ``work``: T * K * (F + 128) floats, of which
    the last one's bits are AR_OK afterwards, AR_ERR_TIMEOUT if a wait ran out."""
    if ids_bytes is None:
        ids_bytes = ids.element_size() if hasattr(ids, "element_size") else 4
    calls = _calls or _layer_calls()
    rc = calls.ar_moe_layer(x, ldx, ids, ids_bytes, w, up, ldup, up_scale, down, lddown,
                            down_scale, out, ldout, work, work_bytes, T, K, E, H, F,
                            DTYPES8.get(dtype, dtype), stream)
    if rc:
        raise ArError(rc, "ar_moe_layer")


class Handle:
    """Owns one handle: ``with Handle(R, N, "bf16") as h: ar_allreduce(h.h, ...)``."""

    def __init__(self, R: int, N: int, dtype):
        self.R, self.N = R, N
        self.dtype = dtype
        self.h = ar_create(R, N, dtype)

    def close(self) -> None:
        if self.h:
            ar_destroy(self.h)
            self.h = 0

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
