"""Launch shapes of the gradients around the experts: every width, number of experts and set of
optional rows that the calls take has CTAs and fits a CTA's shared memory (block_shape.cuh, by a host
program built with nvcc), and on the GPU the widths and k at which a CTA's shared memory is largest.

The bounds are those of test_block."""

import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from test_block import BF, EPS, F32, OPS, SUM, U, Block, Norm, backward, f64, inputs, moe, near, take

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_size_has_a_launch(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    exe = tmp_path / "block_shape_check"
    subprocess.run([nvcc, "-O2", "-std=c++17", "-I", os.path.join(ROOT, "grouped_ffn_gb300", "csrc"),
                    "-o", str(exe), os.path.join(ROOT, "tests", "block_shape_check.cu")],
                   check=True, capture_output=True, timeout=300)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "block shapes ok" in r.stdout


@pytest.fixture(scope="module")
def built():
    from grouped_ffn_gb300 import build
    build.build()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("k", range(9, 16))
@pytest.mark.parametrize("H", [1024, 4096, 7168, 8192, 16384])
def test_gradients_of_many_experts(built, H, k, dt):
    m = moe()
    T = 3
    s = inputs(T, H, k, dt, True, True, True, 0.1, seed=k)
    live = s["dest"].cpu().numpy() >= 0
    for shared in (s["shared"], None):
        q = {**s, "shared": shared}
        out, ws = backward(q, True)
        m.moe_check_device_status(ws)
        want = Block(q, T, H, True, 1.0).backward()
        near(out["rows"][s["dest"][s["dest"] >= 0].long()], want["rows"][0][live], want["rows"][1][live], "rows")
        for name in ("w", "shared", "weight", "gate"):
            near(out[name], *want[name], name)
    terms = take(f64(s["grad"]), s["dest"].cpu().numpy())
    wt, n = f64(s["weight"]), Norm(f64(s["x"]))
    hat, dhat = n.out(np.ones(H))
    sc = m.new_norm_scratch(T, H)
    for add in (s["add"], None):
        u, mag = terms.sum(1), np.abs(terms).sum(1)
        if add is not None:
            u, mag = u + f64(add), mag + np.abs(f64(add))
        du = SUM * mag
        d, dd, _ = n.back(u * wt, np.abs(wt) * du + OPS * np.abs(u * wt))
        for res in (s["gy"], None):
            gx, gw = torch.empty_like(s["x"]), torch.empty(H, device="cuda")
            m.moe_norm_backward(s["grad"], s["x"], s["weight"], EPS, gx, gw, ws, sc, dest_row=s["dest"], add=add,
                                residual_grad=res, residual_scale=0.5)
            m.moe_check_device_status(ws)
            r = 0.0 if res is None else 0.5 * f64(res)
            near(gx, r + d, dd + OPS * (np.abs(r) + np.abs(d)), "x")
            near(gw, (u * hat).sum(0),
                 (du * np.abs(hat) + np.abs(u) * dhat + (T * U + OPS) * np.abs(u * hat)).sum(0), "weight")
