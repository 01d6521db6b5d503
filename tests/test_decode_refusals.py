"""What the calls of a decode step refuse, each before any CUDA call (so these run
without a GPU; the addresses are never dereferenced)."""
import pytest

import all_reduce_reduction_gb300 as ar
from all_reduce_reduction_gb300 import build as cuda_build

A = [0x10000000 * (i + 1) for i in range(16)]       # distinct 16-byte aligned addresses
INVALID, UNSUPPORTED = ar.AR_ERR_INVALID, ar.AR_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def built():
    cuda_build.build()


def _code(fn, **kw):
    try:
        fn(stream=0, **kw)
    except ar.ArError as e:
        return e.code
    return ar.AR_OK


CACHE = dict(kcache=A[0], vcache=A[1], kscale=A[2], vscale=A[3], pages=10, page=16, table=A[4],
             width=5, lens=A[5])


def _move(fn, **kw):
    a = dict(CACHE, k=A[6], v=A[7], offsets=A[8], T=9, B=4, heads=2, D=64, dtype="bf16",
             cache_dtype="e4m3")
    a.update(kw)
    return _code(fn, **a)


# a page of the pool has 2 * 16 * 64 elements, a row 128
CACHE_CHANGES = [
    dict(kcache=None), dict(vcache=None), dict(kscale=None), dict(vscale=None), dict(table=None),
    dict(lens=None), dict(page=0), dict(page=-4), dict(width=0), dict(heads=0), dict(D=0),
    dict(dtype="e4m3"), dict(dtype=5), dict(cache_dtype="fp16"), dict(cache_dtype=7),
    dict(cache_dtype="bf16"), dict(kscale=A[2] + 2), dict(vscale=A[3] + 1), dict(table=A[4] + 2),
    dict(lens=A[5] + 1), dict(ldpage=2047), dict(ldtable=4), dict(ldpage=1 << 62),
    dict(cache_dtype="bf16", kscale=None, vscale=None, kcache=A[0] + 1)]
LIMITS = [dict(D=257), dict(heads=1025), dict(pages=1 << 31), dict(B=1 << 31),
          dict(width=1 << 31), dict(page=1 << 20, width=1 << 11),
          dict(heads=1024, page=1 << 15, D=64)]


@pytest.mark.parametrize("change", CACHE_CHANGES + [
    dict(k=None), dict(v=None), dict(k=A[6] + 1), dict(v=A[7] + 1), dict(offsets=A[8] + 2),
    dict(ldk=127), dict(ldv=1), dict(offsets=None)], ids=str)
def test_move_invalid(change):
    assert _move(ar.ar_cache_write, **change) == INVALID
    assert _move(ar.ar_cache_read, **change) == INVALID


@pytest.mark.parametrize("change", [
    dict(kcache=A[6]), dict(vcache=A[6] + 64), dict(kscale=A[7]), dict(vcache=A[0]),
    dict(vcache=A[0] + 2048), dict(kscale=A[3]), dict(kscale=A[0]), dict(table=A[0] + 16),
    dict(lens=A[1]), dict(offsets=A[2]), dict(kcache=A[4])], ids=str)
def test_write_overlaps(change):
    assert _move(ar.ar_cache_write, **change) == INVALID


@pytest.mark.parametrize("change", [
    dict(k=A[0]), dict(v=A[1] + 16), dict(k=A[7]), dict(v=A[6] + 256), dict(k=A[2]), dict(v=A[3]),
    dict(k=A[4]), dict(v=A[5]), dict(k=A[8])], ids=str)
def test_read_overlaps(change):
    assert _move(ar.ar_cache_read, **change) == INVALID


def test_move_limits():
    for fn in (ar.ar_cache_write, ar.ar_cache_read):
        for change in LIMITS + [dict(T=1 << 31)]:
            assert _move(fn, **change) == UNSUPPORTED, change
        assert _move(fn, T=0) == ar.AR_OK
        assert _move(fn, T=0, B=0, offsets=None, k=None, v=None) == ar.AR_OK
        # pools whose pages alternate in one buffer, rows that are slices of one buffer: no
        # overlap, so the call goes on to the next check
        assert _move(fn, vcache=A[0] + 2048, ldpage=4096, lens=None) == INVALID
        # nothing has a place: no launch
        assert _move(fn, pages=0, kcache=None, vcache=None, kscale=None, vscale=None) == ar.AR_OK
        assert _move(fn, B=0) == ar.AR_OK


def _attend(**kw):
    a = dict(CACHE, q=A[6], scale=0.125, out=A[7], lse=A[8], work=A[9],
             work_bytes=ar.AR_CACHE_WORK_ROWS * 66 * 4, B=4, heads=8, kv_heads=2, D=64,
             dtype="bf16", cache_dtype="e4m3")
    a.update(kw)
    return _code(ar.ar_cache_attention, **a)


@pytest.mark.parametrize("change", [
    {("kv_heads" if k == "heads" else k): v for k, v in c.items()} for c in CACHE_CHANGES] + [
    dict(q=None), dict(out=None), dict(work=None), dict(q=A[6] + 1), dict(out=A[7] + 1),
    dict(lse=A[8] + 2), dict(work=A[9] + 4), dict(work_bytes=ar.AR_CACHE_WORK_ROWS * 66 * 4 - 1),
    dict(ldq=511), dict(ldout=100), dict(heads=9), dict(heads=0), dict(heads=1), dict(out=A[6]),
    dict(out=A[0]), dict(out=A[4]), dict(out=A[8]), dict(lse=A[5]), dict(lse=A[9] + 16),
    dict(work=A[1]), dict(work=A[6]), dict(work=A[3])], ids=str)
def test_attention_invalid(change):
    assert _attend(**change) == INVALID


def test_attention_limits():
    for c in LIMITS:
        c = {("kv_heads" if k == "heads" else k): v for k, v in c.items()}
        assert _attend(**c) == UNSUPPORTED, c
    assert _attend(heads=2048, kv_heads=2) == UNSUPPORTED
    assert _attend(B=0) == ar.AR_OK


def _moe(**kw):
    a = dict(x=A[0], ids=A[1], w=A[2], up=A[3], up_scale=A[4], down=A[5], down_scale=A[6],
             out=A[7], work=A[8], work_bytes=8 * (256 + 128) * 4, T=4, K=2, E=8, H=512, F=256,
             dtype="bf16")
    a.update(kw)
    return _code(ar.ar_moe_layer, **a)


@pytest.mark.parametrize("change", [
    dict(x=None), dict(ids=None), dict(up=None), dict(up_scale=None), dict(down=None),
    dict(down_scale=None), dict(out=None), dict(work=None), dict(x=A[0] + 1), dict(ids=A[1] + 2),
    dict(ids=A[1] + 4, ids_bytes=8), dict(ids_bytes=2), dict(w=A[2] + 2), dict(up_scale=A[4] + 1),
    dict(down_scale=A[6] + 2), dict(out=A[7] + 1), dict(work=A[8] + 4),
    dict(work_bytes=8 * (256 + 128) * 4 - 1), dict(K=0), dict(K=33), dict(E=0), dict(H=0),
    dict(F=0), dict(dtype="e4m3"), dict(dtype=4), dict(ldx=511), dict(ldup=511), dict(lddown=255),
    dict(ldout=511), dict(out=A[0]), dict(out=A[1]), dict(out=A[2]), dict(out=A[3] + 512),
    dict(out=A[4]), dict(out=A[5]), dict(out=A[6]), dict(out=A[8]), dict(work=A[0]),
    dict(work=A[3]), dict(work=A[1]), dict(ldup=1 << 62)], ids=str)
def test_moe_invalid(change):
    assert _moe(**change) == INVALID


def test_moe_limits():
    for c in (dict(E=1025), dict(H=1 << 24), dict(F=1 << 24), dict(T=65), dict(T=64, K=9),
              dict(T=1 << 62)):
        assert _moe(**c) == UNSUPPORTED, c
    assert _moe(T=0) == ar.AR_OK
