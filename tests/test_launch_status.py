"""A launch that the runtime refuses is reported once: the launch helpers leave no error behind that
the thread's next call would report although its kernel runs."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_refused_launches_leave_no_error(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    exe = tmp_path / "launch_status_check"
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-std=c++17", "-Xlinker",
                    "--wrap=cudaLaunchKernelExC,--wrap=cudaGetLastError",
                    "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "grouped_ffn_gb300", "csrc"),
                    "-o", str(exe), os.path.join(ROOT, "tests", "launch_status_check.cu")], check=True, capture_output=True, timeout=300)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "launch status ok" in r.stdout
