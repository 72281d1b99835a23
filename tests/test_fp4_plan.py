"""Host-side check (no GPU) that the plan by which rows are brought to 4 bits leaves no column out:
tests/fp4_plan_check.cu is built with nvcc and walks the plan's spans for every width."""
import os
import subprocess

import pytest

from conftest import ROOT
from test_gemm_schedule import _nvcc


def test_every_span_of_a_row_belongs_to_a_thread(tmp_path):
    nvcc = _nvcc()
    if nvcc is None:
        pytest.skip("nvcc not found")
    exe = tmp_path / "fp4_plan_check"
    cmd = [nvcc, "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a",
           "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "stream_diffusion_transformer_b200", "csrc"),
           os.path.join(ROOT, "tests", "fp4_plan_check.cu"), "-o", str(exe)]
    subprocess.run(cmd, check=True, capture_output=True, text=True, timeout=300)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stdout + out.stderr
    assert out.stdout.split() == ["plan", "ok", str(2 * 7 * 512)], out.stdout
