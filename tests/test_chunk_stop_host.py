"""The stop of the chunk attention's loads, checked on the host: kvk_chunk_stop.cuh is compiled
into a model of a CTA pair's operand ring (tests/stop_check.cpp), which is stopped at random moments
of random schedules."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_a_stop_waits_for_every_load_in_flight_and_for_nothing_else(tmp_path):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("needs g++")
    exe = tmp_path / "stop_check"
    subprocess.run([cxx, "-std=c++17", "-O2", "-I",
                    os.path.join(ROOT, "compressed_decode_attention_kvk_b200", "csrc"),
                    os.path.join(ROOT, "tests", "stop_check.cpp"), "-o", str(exe)],
                   check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout + r.stderr
    assert int(r.stdout.split()[1]) > 10000
