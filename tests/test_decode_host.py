"""The host side of a decode step's calls, on the CPU: where the cache's positions lie,
what the binding makes of its arguments, and the C entry points.  Nothing is launched."""
import os
import shutil
import subprocess
import sys
import sysconfig

import pytest

import all_reduce_reduction_gb300 as ar
from all_reduce_reduction_gb300 import build as cuda_build
from test_layer_threads import PROGRAM

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CALLS = {"ar_cache_write": 23, "ar_cache_read": 23, "ar_cache_attention": 27, "ar_moe_layer": 22}

PLACES = r"""
#include <stdio.h>

#include <vector>

#include "ar_cache.cuh"

using namespace ar;

// every row of calls with good and bad lengths, offsets and tables: the place is that
// of the definition, and every index that leads to it lies in its array
int main() {
    const int bad[] = {-2147483647 - 1, -7, -1, 0, 1, 2, 3, 5, 6, 7, 40, 2147483647};
    long checked = 0, placed = 0;
    for (uint32_t page = 1; page <= 3; ++page)
    for (uint32_t width = 1; width <= 2; ++width)
    for (uint32_t count = 0; count <= 3; ++count)
    for (int n0 : bad)
    for (int n1 : bad)
    for (int o0 : bad)
    for (int o1 : bad)
    for (int o2 : bad)
    for (int with = 0; with < 2; ++with) {
        const int32_t lens[2] = {n0, n1}, offsets[3] = {o0, o1, o2};
        // one word of the table is always outside the pool
        std::vector<int32_t> table = {0, -1, 2, 1};
        table.resize(2 * width);
        Pages g = {};
        g.table = table.data();
        g.lens = lens;
        g.ldtable = width;
        g.count = count;
        g.page = page;
        g.by_page = divide_by(page);
        g.width = width;
        g.heads = 2;
        g.D = 5;
        const uint32_t T = with ? 8 : 2;
        const bool sorted = o0 <= o1 && o1 <= o2;
        for (uint32_t t = 0; t < T; ++t) {
            const int2 at = g.place(with ? offsets : nullptr, 2, t);
            ++checked;
            if (at.x >= 0 && (at.x >= (int)count || at.y < 0 || at.y >= (int)page))
                return printf("outside the pool\n"), 1;
            placed += at.x >= 0;
            if (with && !sorted)
                continue;                       // any place inside the pool will do
            int want = -1, slot = 0;
            for (int b = 0; b < 2; ++b) {
                const long lo = with ? offsets[b] : b, hi = with ? offsets[b + 1] : b + 1;
                if ((long)t < lo || (long)t >= hi)
                    continue;
                long n = lens[b];
                n = n < 0 ? 0 : n > (long)(width * page) ? width * page : n;
                const long j = n - (hi - (long)t);
                if (j >= 0) {
                    want = table[b * width + j / page];
                    slot = j % page;
                }
            }
            if (want < 0 || want >= (int)count)
                want = -1;
            if (at.x != want || (want >= 0 && at.y != slot))
                return printf("row %u at (%d, %d), not (%d, %d)\n", t, at.x, at.y, want, slot), 1;
        }
    }
    // many sequences, empty ones among them: the search against a walk
    for (uint32_t B : {1u, 2u, 31u, 32u, 33u, 34u, 64u, 65u, 1023u, 1024u, 1025u, 1057u, 5000u}) {
        std::vector<int32_t> offsets(B + 1), lens(B, 9), table(B, 0);
        offsets[0] = B % 3;
        for (uint32_t b = 0; b < B; ++b)
            offsets[b + 1] = offsets[b] + (b * 7919u + B) % 4;
        Pages g = {};
        g.table = table.data();
        g.lens = lens.data();
        g.ldtable = 1;
        g.count = 1;
        g.page = 9;
        g.by_page = divide_by(9);
        g.width = 1;
        uint32_t b = 0;
        for (uint32_t t = 0; t < (uint32_t)offsets[B] + 3; ++t) {
            while (b < B && offsets[b + 1] <= (int32_t)t)
                ++b;
            const bool in = b < B && offsets[b] <= (int32_t)t;
            const int2 at = g.place(offsets.data(), B, t);
            if ((at.x == 0) != in || (in && at.y != 9 - (offsets[b + 1] - (int32_t)t)))
                return printf("row %u of %u sequences\n", t, B), 1;
        }
    }
    // the division, at both ends of each quotient's range
    for (uint32_t d = 1; d < 5000; ++d)
        for (uint64_t n = 0; n < 1ull << 31; n = n * 2 + d) {
            const uint64_t q = n / d * d;
            for (uint64_t x : {n, q, q ? q - 1 : q, q + d - 1, (uint64_t)((1u << 31) - 1)})
                if (x < 1ull << 31 && divide_by(d)((uint32_t)x) != x / d)
                    return printf("%llu / %u\n", (unsigned long long)x, d), 1;
        }
    for (uint32_t d : {1u << 30, (1u << 30) + 1, (1u << 31) - 1, 1u << 31})
        for (uint32_t x : {0u, 1u, (1u << 30) - 1, 1u << 30, (1u << 30) + 1, (1u << 31) - 1})
            if (divide_by(d)(x) != x / d)
                return printf("%u / %u\n", x, d), 1;
    // offsets past 32 bits
    Pages g = {};
    g.heads = 1024;
    g.page = 128;
    g.D = 256;
    if (g.scale_at(2000000000, 1023, 127) != 2000000000ull * 1024 * 128 + 1023 * 128 + 127 ||
        g.in_page(1023, 127) != (1023u * 128 + 127) * 256)
        return printf("an offset was cut\n"), 1;
    printf("%ld rows, %ld with a place\n", checked, placed);
    return placed == 0;
}
"""


def test_places_against_the_definition(tmp_path):
    src = tmp_path / "places.cu"
    src.write_text(PLACES)
    exe = str(tmp_path / "places")
    cmd = [cuda_build.nvcc(), *cuda_build.ARCH, "-O1", "-std=c++17", "-I" + cuda_build.INCLUDE,
           "-I" + cuda_build.CSRC, "-Xcompiler", "-fsanitize=address", str(src), "-o", exe]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    res = subprocess.run([exe], capture_output=True, text=True,
                         env=dict(os.environ, ASAN_OPTIONS="protect_shadow_gap=0:detect_leaks=0"))
    assert res.returncode == 0, res.stdout + res.stderr


def test_argument_counts():
    cuda_build.build()
    calls = ar._layer_calls()
    for name, n in CALLS.items():
        assert len(ar.SIGNATURES[name][0]) == n
        for k in (0, n - 1, n + 1):
            with pytest.raises(TypeError):
                getattr(calls, name)(*([0] * k))


class _Recorder:
    """Stands in for the extension module; keeps what a call was given."""

    def __getattr__(self, name):
        def call(*args):
            self.args = args
            return ar.AR_OK
        return call


def test_what_the_binding_passes(monkeypatch):
    """Every argument at its place, and the defaults."""
    rec = _Recorder()
    monkeypatch.setattr(ar, "_calls", rec)
    ar.ar_cache_write("k", "v", "kc", "vc", "ks", "vs", 7, 16, "table", 5, "lens", "off", 3, 2, 4,
                      64, "fp16", ldk=1, ldv=2, ldpage=3, ldtable=4, stream="s")
    assert rec.args == ("k", 1, "v", 2, "kc", "vc", 3, "ks", "vs", 7, 16, "table", 4, 5, "lens",
                        "off", 3, 2, 4, 64, ar.AR_FP16, ar.AR_FP16, "s")
    ar.ar_cache_read("kc", "vc", "ks", "vs", 7, 16, "table", 5, "lens", "off", "k", "v", 3, 2, 4,
                     64, "bf16", "e4m3", ldk=1, ldv=2, ldpage=3, ldtable=4)
    assert rec.args == ("kc", "vc", 3, "ks", "vs", 7, 16, "table", 4, 5, "lens", "off", "k", 1,
                        "v", 2, 3, 2, 4, 64, ar.AR_BF16, ar.AR_E4M3, None)
    ar.ar_cache_attention("q", "kc", "vc", "ks", "vs", 7, 16, "table", 5, "lens", 0.5, "out",
                          "lse", "work", 99, 2, 8, 4, 64, "bf16", "e4m3", window=6, ldq=1,
                          ldpage=2, ldtable=3, ldout=4)
    assert rec.args == ("q", 1, "kc", "vc", 2, "ks", "vs", 7, 16, "table", 3, 5, "lens", 0.5, 6,
                        "out", 4, "lse", "work", 99, 2, 8, 4, 64, ar.AR_BF16, ar.AR_E4M3, None)
    ar.ar_moe_layer("x", 123, "w", "up", "us", "down", "ds", "out", "work", 99, 1, 2, 3, 4, 5,
                    "fp32", ldx=6, ldup=7, lddown=8, ldout=9)
    assert rec.args == ("x", 6, 123, 4, "w", "up", 7, "us", "down", 8, "ds", "out", 9, "work", 99,
                        1, 2, 3, 4, 5, ar.AR_FP32, None)

    class Ids:
        def element_size(self):
            return 8
    ar.ar_moe_layer("x", Ids(), "w", "up", "us", "down", "ds", "out", "work", 99, 1, 2, 3, 4, 5,
                    "fp32")
    assert rec.args[3] == 8


# every call waits until the other thread has moved on, three seconds at most
STAND_IN = r"""
#include <unistd.h>
volatile long ar_test_count;
static int blocked(void) {
    const long from = ar_test_count;
    for (int i = 0; i < 3000 && ar_test_count == from; ++i)
        usleep(1000);
    return ar_test_count == from ? 99 : 0;
}
""" + "".join("int %s() { return blocked(); }\n" % n for n in ar.SIGNATURES
              if n in CALLS or n.startswith(("ar_rmsnorm", "ar_moe", "ar_matmul8")))


@pytest.fixture(scope="module")
def stand_in(tmp_path_factory):
    at = tmp_path_factory.mktemp("stand_in")
    (at / "stand_in.c").write_text(STAND_IN)
    lib, module = str(at / "libar_gb300.so"), str(at / "_native.so")
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", lib, str(at / "stand_in.c")], check=True)
    subprocess.run(["gcc", "-shared", "-fPIC", "-O2", "-I" + cuda_build.INCLUDE,
                    "-I/usr/local/cuda/include", "-I" + sysconfig.get_paths()["include"],
                    cuda_build.NATIVE_SOURCE, "-o", module, "-L" + str(at), "-lar_gb300",
                    "-Wl,-rpath," + str(at)], check=True)
    return lib, module


@pytest.mark.parametrize("name", sorted(CALLS))
def test_other_threads_run_while_a_call_blocks(stand_in, name):
    res = subprocess.run([sys.executable, "-c", PROGRAM, *stand_in, name, str(CALLS[name])],
                         capture_output=True, text=True, timeout=60, env=dict(os.environ))
    assert res.returncode == 0, res.stderr
    assert res.stdout.strip() == "0"


C_PROGRAM = r"""
#include "ar.h"

int main(void) {
    const void *x = 0;
    void *y = 0;
    float *f = 0;
    int32_t *i = 0;
    int rc = ar_cache_write(x, 0, x, 0, y, y, 0, f, f, 8, 64, i, 0, 4, i, i, 2, 2, 8,
                            AR_CACHE_MAX_DIM, AR_BF16, AR_E4M3, 0);
    rc |= ar_cache_read(x, x, 0, f, f, 8, 64, i, 0, 4, i, i, y, 0, y, 0, 2, 2,
                        AR_CACHE_MAX_HEADS, 128, AR_BF16, AR_E4M3, 0);
    rc |= ar_cache_attention(x, 0, x, x, 0, f, f, 8, 64, i, 0, 4, i, 1.0f, 0, y, 0, f, f,
                             AR_CACHE_WORK_ROWS * (128 + 2) * sizeof(float), 2, 16, 8, 128,
                             AR_BF16, AR_E4M3, 0);
    rc |= ar_moe_layer(x, 0, i, 4, f, x, 0, f, x, 0, f, y, 0, f,
                       AR_MOE_LAYER_PAIRS * (256 + 128) * sizeof(float), AR_MOE_LAYER_TOKENS, 8,
                       64, 512, 256, AR_BF16, 0);
    return rc;
}
"""


@pytest.mark.skipif(shutil.which("gcc") is None, reason="no C compiler")
def test_entry_points_link_from_c11(tmp_path):
    lib = cuda_build.build()
    src = tmp_path / "decode.c"
    src.write_text(C_PROGRAM)
    cmd = ["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror", "-pedantic",
           "-I" + os.path.join(ROOT, "include"), "-I/usr/local/cuda/include", str(src), "-o",
           str(tmp_path / "decode"), "-L" + os.path.dirname(lib), "-lar_gb300",
           "-Wl,-rpath," + os.path.dirname(lib)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
