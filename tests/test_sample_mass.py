"""The fixed-point scale of the samplers' masses, checked on the CPU: the sums
of every accepted vocabulary stay below 2^64 (tests/cpp/sample_mass_check.cu),
and draws from equal masses of that scale are those of the definition."""
import os
import subprocess
import tempfile

import pytest

from test_work_split import ROOT, _nvcc


def test_masses_of_every_vocabulary_fit():
    nvcc = _nvcc()
    if nvcc is None:
        pytest.skip("nvcc not available")
    with tempfile.TemporaryDirectory() as d:
        exe = os.path.join(d, "sample_mass_check")
        r = subprocess.run([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_100a,code=sm_100a",
                            os.path.join(ROOT, "tests", "cpp", "sample_mass_check.cu"), "-o", exe],
                           capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, r.stderr[-4000:]
        out = subprocess.run([exe], capture_output=True, text=True, timeout=600)
        assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout[-2000:] + out.stderr[-2000:]


def test_equal_masses_of_the_widest_row():
    """u * (kept mass) and its borders in the kernel's arithmetic (fp64 product,
    truncated), 2^18 tokens of 2^45: the token is floor(u * 2^18)."""
    V, unit = 1 << 18, 1 << 45
    for n in list(range(0, 1 << 24, 65521)) + [1 << 23, (1 << 24) - 1, 64, 63, 65, 3 << 22]:
        u = n / (1 << 24)                              # every fp32 uniform is such a fraction or finer
        target = int(u * float(V * unit))
        assert target // unit == n * V >> 24
