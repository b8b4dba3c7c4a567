"""The paged attention and the row sampler on a second device of one process,
without a GPU: their launchers run over a stand-in for the CUDA runtime
(tests/cpp/two_devices_check.cpp) that refuses a launch whose shared memory the
current device has not been asked for."""
import os
import shutil
import subprocess
import tempfile

import pytest

from test_work_split import ROOT, _nvcc


def test_launchers_on_a_second_device():
    nvcc, cxx = _nvcc(), shutil.which("g++")
    if nvcc is None or cxx is None:
        pytest.skip("no compiler")
    from decoder_only_transformer_llama_b200 import build as B
    B.build()                                              # the object files, if they are not there yet
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    objs = [os.path.join(B.BUILD, n + ".o") for n in ("paged_attention", "paged_attention_tile", "sample_rows")]
    with tempfile.TemporaryDirectory() as d:
        exe = os.path.join(d, "two_devices_check")
        r = subprocess.run([cxx, "-std=c++17", "-O1", "-I", include,
                            os.path.join(ROOT, "tests", "cpp", "two_devices_check.cpp"), *objs, "-o", exe, "-lpthread"],
                           capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stderr[-4000:]
        out = subprocess.run([exe], capture_output=True, text=True, timeout=60)
        assert out.returncode == 0 and out.stdout.strip().endswith("ok"), out.stdout[-2000:] + out.stderr[-2000:]
