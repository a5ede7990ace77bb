"""Host side of the gradient operators over a fake CUDA runtime (tests/c/fake_cudart.cpp): no GPU, no device work."""
import os
import shutil
import subprocess

import pytest

from collective_communication_schedules_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HERE = os.path.join(ROOT, "tests", "c")


@pytest.mark.skipif(shutil.which("g++") is None, reason="no C++ compiler")
def test_tensor_lists(tmp_path):
    out = str(tmp_path / "tensor_list")
    cmd = [build.nvcc()] + build.ARCH + ["-O1", "-std=c++17", "-cudart", "none", "-I", build.INCLUDE, "-I", build.CSRC,
                                         "-I", HERE, os.path.join(HERE, "tensor_list.cpp"),
                                         os.path.join(HERE, "fake_cudart.cpp"), os.path.join(build.CSRC, "grad.cu"), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([out], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and "LISTS OK" in r.stdout, r.stdout + r.stderr
