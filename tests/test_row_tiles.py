"""How the FP4 product cuts a segment's rows into tiles (row_tile of
grouped_ffn_gb300/csrc/tile_order.cuh), up to the largest segment.  Checked by
a host program built with nvcc from the header the kernel uses, and on the GPU
at the largest size."""

import os
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_row_tiles_cover_a_segment(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    exe = tmp_path / "row_tile_check"
    subprocess.run([nvcc, "-O2", "-std=c++17", "-I", os.path.join(ROOT, "grouped_ffn_gb300", "csrc"),
                    "-o", str(exe), os.path.join(ROOT, "tests", "row_tile_check.cu")],
                   check=True, capture_output=True, timeout=300)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "row tiles ok" in r.stdout


@pytest.mark.gpu
def test_largest_segment():
    """One segment of 2^31 - 17 rows: its ends and its middle against the same rows alone."""
    from grouped_ffn_gb300 import build, moe as m
    build.build()
    n, N, K = 2 ** 31 - 17, 8, 32                       # 34 GB of codes, 17 GB of scales, 34 GB of results
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    wc = torch.randint(0, 256, (1, N, K // 2), generator=gen, device="cuda").to(torch.uint8)
    ld = m.moe_fp4_scale_ld(K, m.MOE_FP4_MX)
    wsf = torch.zeros(1, N, ld, dtype=torch.uint8, device="cuda")
    wsf[:, :, 0] = 127
    w = m.pack_weights_fp4(wc, wsf, m.MOE_FP4_MX, m.MOE_EPI_NONE)
    xc = torch.randint(0, 256, (900, K // 2), generator=gen, device="cuda").to(torch.uint8)
    xs = torch.zeros(900, ld, dtype=torch.uint8, device="cuda")
    xs[:, 0] = 127
    places = [slice(0, 300), slice(n // 2, n // 2 + 300), slice(n - 300, n)]
    codes, sf = m.new_fp4(n, K, m.MOE_FP4_MX)
    codes.zero_(), sf.zero_()
    sf[:, 0] = 127
    for i, p in enumerate(places):
        codes[p] = xc[300 * i:300 * i + 300]
    ws = m.new_workspace(1, 1, 1)
    expert = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((n, N), 3.0, dtype=torch.bfloat16, device="cuda")
    m.moe_grouped_product_fp4(codes, sf, torch.tensor([0, n], dtype=torch.int32, device="cuda"), expert, w, None, out,
                              ws)
    m.moe_check_device_status(ws)
    few = torch.empty(900, N, dtype=torch.bfloat16, device="cuda")
    m.moe_grouped_product_fp4(xc, xs, torch.tensor([0, 900], dtype=torch.int32, device="cuda"), expert, w, None, few,
                              ws)
    assert few.abs().max() > 0
    for i, p in enumerate(places):
        assert torch.equal(out[p], few[300 * i:300 * i + 300])
        out[p] = 0
    for lo in range(0, n, 1 << 27):
        assert not out[lo:lo + (1 << 27)].any()
