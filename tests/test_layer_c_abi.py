"""The layer operators' entry points from C11 (compile and link only; nothing is
run, so no GPU is needed)."""
import os
import shutil
import subprocess

import pytest

from all_reduce_reduction_gb300 import build as cuda_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

C_PROGRAM = r"""
#include "ar.h"

int main(void) {
    const void *x = 0;
    void *y = 0;
    float *f = 0;
    int32_t *i = 0;
    int rc = ar_rmsnorm(x, 0, x, 0, x, 1e-6f, y, 0, y, 0, f, f, 4, AR_SCALE_BLOCK, AR_BF16,
                        AR_E4M3, 0);
    rc |= ar_rmsnorm_grad(x, 0, x, 0, x, 0, x, f, y, 0, f, f,
                          AR_NORM_GRAD_ROWS * AR_SCALE_BLOCK * sizeof(float), 4, AR_SCALE_BLOCK,
                          AR_BF16, 0);
    rc |= ar_moe_route(x, 4, 4, AR_MOE_MAX_CHOICES, AR_MOE_MAX_EXPERTS, i, i, i, 0);
    rc |= ar_moe_dispatch(x, 0, f, i, y, 0, f, 8, 4, 2, 128, AR_E4M3, 0);
    rc |= ar_moe_return(x, 0, 8, i, f, y, 0, 4, 2, 128, AR_FP32, 0);
    rc |= ar_moe_return_grad(x, 0, x, 0, 8, i, f, y, 0, f, 4, 2, 128, AR_FP16, 0);
    rc |= ar_matmul8(x, 0, f, x, 0, f, i, 2, y, 0, 8, 128, 128, AR_BF16, i, 0);
    return rc;
}
"""


@pytest.mark.skipif(shutil.which("gcc") is None, reason="no C compiler")
def test_layer_entry_points_link_from_c11(tmp_path):
    lib = cuda_build.build()
    src = tmp_path / "layer.c"
    src.write_text(C_PROGRAM)
    cmd = ["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror", "-pedantic",
           "-I" + os.path.join(ROOT, "include"), "-I/usr/local/cuda/include", str(src), "-o",
           str(tmp_path / "layer"), "-L" + os.path.dirname(lib), "-lar_gb300",
           "-Wl,-rpath," + os.path.dirname(lib)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
