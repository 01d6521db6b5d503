"""Which buffers the layer operators take as overlapping: the check against every
byte of small matrices.  Compiled and run on the host, no GPU needed."""
import os
import subprocess

from all_reduce_reduction_gb300 import build as cuda_build

PROGRAM = r"""
#include <stdio.h>

#include <set>

#include "ar_rows.cuh"

using namespace ar;

// the bytes of the matrix
static std::set<uintptr_t> bytes(uintptr_t p, size_t ld, size_t rows, size_t cols) {
    std::set<uintptr_t> s;
    for (size_t r = 0; r < rows; ++r)
        for (size_t c = 0; c < cols; ++c)
            s.insert(p + r * ld + c);
    return s;
}

int main() {
    long checked = 0, apart = 0, missed = 0, refused = 0;
    for (size_t ra = 0; ra <= 3; ++ra)
    for (size_t rb = 0; rb <= 3; ++rb)
    for (size_t ca = 1; ca <= 4; ++ca)
    for (size_t cb = 1; cb <= 4; ++cb)
    for (size_t la = ca; la <= 7; ++la)
    for (size_t lb = cb; lb <= 7; ++lb)
    for (uintptr_t pb = 80; pb <= 120; ++pb) {
        const Matrix a = matrix((const void *)100, la, ra, ca, 1);
        const Matrix b = matrix((const void *)pb, lb, rb, cb, 1);
        const std::set<uintptr_t> x = bytes(100, la, ra, ca);
        bool share = false;
        for (uintptr_t q : bytes(pb, lb, rb, cb))
            share = share || x.count(q);
        const bool said = meet(a, b);
        if (said != meet(b, a))
            return printf("not symmetric\n"), 1;
        ++checked;
        apart += !share;
        missed += share && !said;
        // slices of one buffer: no byte shared, one stride, rows whole within it
        const uintptr_t in = pb >= 100 ? (pb - 100) % la : la - (100 - pb) % la;
        if (la == lb && ra > 1 && rb > 1 && in >= ca && in + cb <= la && said)
            ++refused;
        // exactly the same matrix, rows of one length: one row has no stride
        if (ra == rb && ca == cb && pb == 100 && (la == lb || ra <= 1) && !same(a, b))
            return printf("the same matrix not seen\n"), 1;
        if (ra == rb && ca == cb && ra > 1 && (la != lb || pb != 100) && same(a, b))
            return printf("another matrix taken as the same\n"), 1;
    }
    printf("%ld pairs, %ld apart, %ld overlaps missed, %ld slices refused\n", checked, apart,
           missed, refused);
    return missed || refused;
}
"""


def test_meet_against_every_byte(tmp_path):
    src = tmp_path / "overlap.cu"
    src.write_text(PROGRAM)
    exe = str(tmp_path / "overlap")
    cmd = [cuda_build.nvcc(), *cuda_build.ARCH, "-std=c++17", "-I" + cuda_build.INCLUDE,
           "-I" + cuda_build.CSRC, str(src), "-o", exe]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    res = subprocess.run([exe], capture_output=True, text=True, env=dict(os.environ))
    assert res.returncode == 0, res.stdout
