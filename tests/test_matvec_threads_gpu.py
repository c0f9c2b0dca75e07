"""Host threads that share one kernel of the product from codes, without an interpreter lock between
them: tests/c/matvec_threads.c, compiled and run."""
import os
import shutil
import subprocess

import pytest

from quantized_zero_communication_gb300 import build as zbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
def test_threads_share_a_kernel(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    libdir, exe = os.path.dirname(zbuild.build()), str(tmp_path / "threads")
    r = subprocess.run(
        ["gcc", "-std=gnu11", "-O2", "-Wall", os.path.join(ROOT, "tests", "c", "matvec_threads.c"),
         "-I", os.path.join(ROOT, "include"), "-I", os.path.join(cuda, "include"), "-L", libdir, "-lzpp",
         "-L", os.path.join(cuda, "lib64"), "-lcudart", "-lpthread", f"-Wl,-rpath,{libdir}",
         f"-Wl,-rpath,{os.path.join(cuda, 'lib64')}", "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "threads OK" in r.stdout, r.stdout + r.stderr
