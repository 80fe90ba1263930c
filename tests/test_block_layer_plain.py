"""A layer with a block whose last step had no residual: that step is the plain weighted sum, and so
is its gradient (the same bits as the call on the step's own buffers)."""

import pytest
import torch

from test_block import BF
from test_block_layer import make, moe


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_ffn_gb300 import build
    build.build()


@pytest.mark.gpu
@pytest.mark.parametrize("shared", [False, True])
def test_gradient_of_a_step_without_residual(shared):
    m = moe()
    T, H, I, E, k = 21, 256, 128, 8, 3
    layer, d = make(T, H, I, E, k, shared)
    n, y = torch.empty(T, H, dtype=BF, device="cuda"), torch.empty(T, H, device="cuda")
    plain = torch.empty(T, H, dtype=BF, device="cuda")
    m.moe_norm(d["x"], d["pre"], 1e-6, n)
    layer.forward(d["logits"], n, y, residual=d["x"], gate=d["gate"])
    layer.forward(d["logits"], n, plain)
    gy = d["rn"](T, H)
    new = lambda: (torch.zeros(T * k, H, dtype=BF, device="cuda"), torch.zeros(T, k, device="cuda"))
    (rows, gw), (rows2, gw2), (rows3, gw3) = new(), new(), new()
    layer.combine_backward(gy, rows, gw)
    layer.check()
    m.moe_combine_backward(gy, layer.y_perm[:T * k], layer.dest_row[:T * k], layer.topk_w[:T], rows2, gw2, layer.ws)
    assert torch.equal(rows, rows2) and torch.equal(gw, gw2)
    for bad in (dict(gate=d["gate"]), dict(grad_weight=torch.empty(H, device="cuda")),
                dict(grad_gate=torch.empty(T, device="cuda"))):
        with pytest.raises(ValueError):
            layer.combine_backward(gy, rows, gw, **bad)
    # and through norm and gate again after a step with a residual
    layer.forward(d["logits"], n, y, residual=d["x"], gate=d["gate"])
    layer.combine_backward(gy, rows, gw, gate=d["gate"])
    m.moe_combine_norm_backward(gy, layer.y_perm[:T * k], layer.dest_row[:T * k], layer.topk_w[:T], layer.block,
                                rows3, gw3, layer.ws, shared=layer.shared_output(T), weight=layer.post_weight,
                                gate=d["gate"])
    assert torch.equal(rows, rows3) and torch.equal(gw, gw3) and not torch.equal(rows, rows2)


@pytest.mark.gpu
def test_steps_of_both_kinds_in_graphs():
    """Where a replayed step may have been of the other kind than the last forward, the call says which."""
    m = moe()
    T, H, I, E, k = 9, 256, 128, 8, 2
    layer, d = make(T, H, I, E, k)
    n, y = torch.empty(T, H, dtype=BF, device="cuda"), torch.empty(T, H, device="cuda")
    plain, gy = torch.empty(T, H, dtype=BF, device="cuda"), d["rn"](T, H)
    m.moe_norm(d["x"], d["pre"], 1e-6, n)
    new = lambda: (torch.zeros(T * k, H, dtype=BF, device="cuda"), torch.zeros(T, k, device="cuda"))
    layer.forward(d["logits"], n, y, residual=d["x"])
    (rows, gw), (rows2, gw2), (rows3, gw3) = new(), new(), new()
    layer.combine_backward(gy, rows, gw)
    graph = layer.capture(d["logits"], n, y, residual=d["x"])
    layer.forward(d["logits"], n, plain)
    with pytest.raises(ValueError):
        layer.combine_backward(gy, rows2, gw2)
    graph.replay()
    layer.combine_backward(gy, rows2, gw2, residual=True)
    assert torch.equal(rows, rows2) and torch.equal(gw, gw2)
    layer.combine_backward(gy, rows2, gw2, residual=False)
    m.moe_combine_backward(gy, layer.y_perm[:T * k], layer.dest_row[:T * k], layer.topk_w[:T], rows3, gw3, layer.ws)
    assert torch.equal(rows3, rows2) and torch.equal(gw3, gw2)
