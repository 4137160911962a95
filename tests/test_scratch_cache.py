"""The decodes' scratch cache over a fake of the CUDA calls that it makes (CPU)."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_uses_of_a_buffer_wait_for_one_another_also_after_errors(tmp_path):
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    if not os.path.exists(os.path.join(cuda, "cuda.h")):
        pytest.skip("needs the CUDA headers")
    exe = str(tmp_path / "scratch")
    subprocess.run(["g++", "-std=c++17", "-w", "-I", os.path.join(ROOT, "attention_forward_sm_gb300", "csrc"),
                    "-I", cuda, os.path.join(ROOT, "tests", "scratch_host.cpp"), "-o", exe], check=True)
    res = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert res.returncode == 0, res.stdout
