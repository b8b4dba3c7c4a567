"""The work list of the paged attention, checked on the CPU: paged_work.cuh is
host and device code; tests/cpp/paged_work_check.cu walks it against plain
loops (tile and unit counts, the tile of every unit, equal runs for every
number of CTAs)."""
import os
import subprocess
import tempfile

import pytest

from test_work_split import ROOT, _nvcc


def test_paged_work_list():
    nvcc = _nvcc()
    if nvcc is None:
        pytest.skip("nvcc not available")
    with tempfile.TemporaryDirectory() as d:
        exe = os.path.join(d, "paged_work_check")
        r = subprocess.run([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_100a,code=sm_100a",
                            "-I", os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "cpp", "paged_work_check.cu"),
                            "-o", exe], capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, r.stderr[-4000:]
        out = subprocess.run([exe], capture_output=True, text=True, timeout=600)
        assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout[-2000:] + out.stderr[-2000:]
