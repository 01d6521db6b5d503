"""The extension module leaves other Python threads running while a launch blocks:
against a stand-in for the library whose calls wait for one of them.  No GPU."""
import os
import subprocess
import sys
import sysconfig

import pytest

from all_reduce_reduction_gb300 import build as cuda_build

CALLS = {"ar_rmsnorm": 17, "ar_rmsnorm_grad": 17, "ar_moe_route": 9, "ar_moe_dispatch": 13,
         "ar_moe_return": 12, "ar_moe_return_grad": 15, "ar_matmul8": 16}

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
""" + "".join("int %s() { return blocked(); }\n" % n for n in CALLS)

PROGRAM = r"""
import ctypes, importlib.util, sys, threading
from importlib.machinery import ExtensionFileLoader
lib = ctypes.CDLL(sys.argv[1])
count = ctypes.c_long.in_dll(lib, "ar_test_count")
spec = importlib.util.spec_from_loader("_native", ExtensionFileLoader("_native", sys.argv[2]))
calls = importlib.util.module_from_spec(spec)
spec.loader.exec_module(calls)
done = threading.Event()
def other():
    while not done.wait(0.01):
        count.value += 1
thread = threading.Thread(target=other, daemon=True)
thread.start()
name, n = sys.argv[3], int(sys.argv[4])
print(getattr(calls, name)(*([0] * n)))
done.set()
"""


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
