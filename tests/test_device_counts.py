"""Counts that the library asks the driver for once per device (clusters resident at
once) keep an answer of 0 as 0, so that a cluster size that does not fit is not taken."""
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(ROOT, "mixture_experts_routing_gb300", "csrc")
CUDA = next((d for d in (os.environ.get("CUDA_HOME"), "/usr/local/cuda") if d and os.path.exists(os.path.join(d, "include", "cuda_runtime.h"))), None)


@pytest.mark.skipif(shutil.which("g++") is None or CUDA is None, reason="needs g++ and the CUDA headers")
def test_a_count_of_zero_stays_zero(tmp_path):
    exe = str(tmp_path / "check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, "-I", os.path.join(CUDA, "include"), "-o", exe,
                    os.path.join(HERE, "count_per_device_check.cpp"), "-pthread"], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0, out.stdout


@pytest.mark.parametrize("source", ["shared.cu", "shared_few.cu"])
def test_cluster_queries_keep_their_zeros(source):
    with open(os.path.join(CSRC, source)) as f:
        text = f.read()
    body = text[text.index("int max_clusters("):]
    body = body[: body.index("\n}\n")]
    assert "count_per_device(" in body and "cudaOccupancyMaxActiveClusters" in body and "once_per_device" not in body
