"""The microscaled formats used from a plain C program: tests/capi/mx_from_c.c is
compiled with gcc against include/zs.h, linked to libzs.so and the HIP runtime, and run
on the GPU."""
import os
import subprocess
import tempfile

import pytest

import sharded_mixed_precision_shard_amd as zs
from tests.test_gpu_capi import ROCM, ROOT

pytestmark = pytest.mark.gpu


def test_linear_layer_from_c():
    lib_dir = os.path.dirname(zs.LIB_PATH)
    with tempfile.TemporaryDirectory() as d:
        exe = os.path.join(d, "mx_from_c")
        subprocess.run(["gcc", "-std=c11", "-O1", "-D__HIP_PLATFORM_AMD__",
                        "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROCM, "include"),
                        "-o", exe, os.path.join(ROOT, "tests", "capi", "mx_from_c.c"),
                        "-L", lib_dir, "-lzs", "-L", os.path.join(ROCM, "lib"), "-lamdhip64",
                        "-Wl,-rpath," + lib_dir, "-Wl,-rpath," + os.path.join(ROCM, "lib")],
                       check=True, capture_output=True, text=True)
        r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "microscaled: exact" in r.stdout
