"""Which kernel a chunk call takes, checked on the host: kvk_chunk_route.cuh is compiled into a small
program (tests/route_check.cpp).  A tensor-core kernel that was built with other registers than it
hands around leaves its calls to the CUDA-core kernel; it does not fail them."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_chunk_route(tmp_path):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("needs g++")
    exe = tmp_path / "route_check"
    subprocess.run([cxx, "-std=c++17", "-O2", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "compressed_decode_attention_kvk_b200", "csrc"),
                    os.path.join(ROOT, "tests", "route_check.cpp"), "-o", str(exe)],
                   check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout + r.stderr
