"""The rings of ar_moe_layer on the CPU: the steps' stages and phases, and that after a wait
that gave up every copy on its way is waited for.  Nothing is launched."""
import os
import subprocess

from all_reduce_reduction_gb300 import build as cuda_build

PROGRAM = r"""
#include <stdio.h>

#include <vector>

#include "ar_ring.cuh"

using namespace ar;

// A barrier of a stage: phases that have ended, and whether the next one has begun.
struct Barrier {
    uint32_t ended = 0;
    bool open = false;
    bool test(uint32_t parity) const { return (ended & 1) != parity; }
};

// A warp that sends `total` steps through its ring and waits for each in turn.  The copies up
// to `landed` arrive when they are waited for, the later ones not before the end; the first
// wait for one of those gives up, and nothing is sent after it.
static int run(uint32_t bits, uint32_t total, uint32_t landed) {
    const uint32_t stages = 1u << bits;
    std::vector<Barrier> bar(stages);
    RingSteps r = {bits, 0u, 0u};
    bool failed = false;
    uint32_t planned = 0;
    auto send = [&] {
        if (planned == total)
            return 0;
        ++planned;
        if (failed)
            return 0;
        Barrier &b = bar[r.stage(r.sent)];
        if (b.open || (b.ended & 1) != r.parity(r.sent))
            return printf("a stage that is not free\n"), 1;
        b.open = true;
        ++r.sent;
        return 0;
    };
    for (uint32_t i = 0; i < stages; ++i)
        if (send())
            return 1;
    for (uint32_t step = 0; step < total; ++step) {
        Barrier &b = bar[r.stage(r.used)];
        if (!failed && b.test(r.parity(r.used)))
            return printf("a phase that had ended before its copy\n"), 1;
        if (!failed && step < landed) {
            b.open = false;
            ++b.ended;
            if (!b.test(r.parity(r.used)))
                return printf("a wait for another phase\n"), 1;
        } else {
            failed = true;
        }
        ++r.used;
        if (send())
            return 1;
    }
    uint32_t open = 0, waited = 0;
    for (const Barrier &b : bar)
        open += b.open;
    for (uint32_t step = r.oldest_open(); step != r.sent; ++step) {
        Barrier &b = bar[r.stage(step)];
        if (!b.test(r.parity(step))) {           // waits, until it lands
            b.open = false;
            ++b.ended;
            ++waited;
        }
    }
    for (const Barrier &b : bar)
        if (b.open)
            return printf("%u stages, %u steps, %u landed: a copy is left on its way\n", stages,
                          total, landed), 1;
    if (waited != open)
        return printf("waited for %u of %u copies\n", waited, open), 1;
    return 0;
}

int main() {
    for (uint32_t bits = 0; bits <= 2; ++bits)
        for (uint32_t total = 0; total <= 40; ++total)
            for (uint32_t landed = 0; landed <= total; ++landed)
                if (run(bits, total, landed))
                    return 1;
    return 0;
}
"""


def test_every_copy_on_its_way_is_waited_for(tmp_path):
    src = tmp_path / "ring.cu"
    src.write_text(PROGRAM)
    exe = str(tmp_path / "ring")
    res = subprocess.run([cuda_build.nvcc(), *cuda_build.ARCH, "-O1", "-std=c++17",
                          "-I" + cuda_build.CSRC, str(src), "-o", exe], capture_output=True,
                         text=True)
    assert res.returncode == 0, res.stderr
    res = subprocess.run([exe], capture_output=True, text=True, env=dict(os.environ))
    assert res.returncode == 0, res.stdout + res.stderr
