"""The layer with a gate of a balance bias and FP4 experts: each step of
MoELayer.forward against its definition on the step's own inputs (the hidden
rows as the layer holds them), the whole step against its graph, and a
router training step through the layer.

Tolerances: a product of FP4 values as in test_fp4_product; the combine adds k
products in fp32, k + 1 half steps of fp32 of the terms' magnitudes, and one
bf16 rounding, 2^-8 of the value.
"""

import numpy as np
import pytest
import torch

import test_gate as tg
import workloads as wl
from test_fp4_product import product
from test_fp4_rows import MX, NV, reference

pytestmark = pytest.mark.gpu


def moe():
    from grouped_ffn_gb300 import moe as m
    return m


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_ffn_gb300 import build
    build.build()
    torch.cuda.set_device(0)


def values(t, fmt, exp):
    return reference(t.float().cpu().numpy().reshape(-1, t.shape[-1]), fmt, exp)[2].reshape(t.shape)


def expert_values(w, fmt):
    """Weights as the layer holds them: per-expert tensor scale, FP4 values."""
    from grouped_ffn_gb300 import MoELayer
    out = np.empty(w.shape)
    exps = MoELayer._quantize_experts(w, fmt)[2]
    for e, x in enumerate(exps):
        out[e] = values(w[e], fmt, x)
    return out


def near(got, y, err):
    got = got.float().cpu().numpy().astype(np.float64)
    bad = np.abs(got - y) > err + 2 * 2.0 ** -8 * np.abs(y) + 2.0 ** -100
    assert not bad.any(), np.abs(got - y)[bad].max()


@pytest.mark.parametrize("fmt,shared", [(MX, False), (NV, True), (MX, True)])
def test_step(fmt, shared):
    from grouped_ffn_gb300 import MoELayer
    m = moe()
    w = wl.WORKLOADS["tiny"].scaled(T=37, H=512, I=160, E=16, k=3, zipf_s=1.0)
    dev = torch.device("cuda:0")
    pl = wl.make_placement(w)
    logits, x = wl.make_logits(w, dev), wl.make_x(w, dev)
    gen = torch.Generator(device=dev)
    gen.manual_seed(4)
    rnd = lambda *s: (0.05 * torch.randn(*s, generator=gen, device=dev)).bfloat16()
    wgu, wd = rnd(w.E, 2 * w.I, w.H), rnd(w.E, w.H, w.I)
    sgu, sd = (rnd(1, 2 * w.I, w.H), rnd(1, w.H, w.I)) if shared else (None, None)
    bias = 0.1 * torch.randn(w.E, generator=gen, device=dev)
    cfg = m.GateCfg(m.MOE_SCORE_SIGMOID, w.k, 4, 2, 2, 1, 1.5)
    layer = MoELayer(H=w.H, I=w.I, E=w.E, k=w.k, placement=m.DevicePlacement.from_tables(pl, dev),
                     w_gate_up=wgu, w_down=wd, max_tokens=w.T + 3, shared_w_gate_up=sgu, shared_w_down=sd, device=dev,
                     gate=cfg, gate_bias=bias.clone(), fp4=fmt)
    y = torch.empty(w.T, w.H, dtype=torch.bfloat16, device=dev)
    layer.forward(logits, x, y)
    layer.check()
    A = w.T * w.k
    rows = A + (w.T if shared else 0)
    ids, wts = tg.reference(logits.cpu().numpy().astype(np.float64), bias.cpu().numpy(), 1, w.k, 4, 2, 2, True, 1.5)
    assert np.array_equal(layer.topk_ids[:w.T].cpu().numpy(), ids)
    tw = layer.topk_w[:w.T].cpu().numpy().astype(np.float64)
    assert (np.abs(tw - wts) <= 16 * 2.0 ** -24 * wts).all()
    # gate/up: the dispatched rows' values, then the hidden rows
    src = layer.src_assign[:A].cpu().numpy() // w.k
    if shared:
        src = np.concatenate((src, np.arange(w.T)))
    bounds = layer.seg_offsets.cpu().numpy()
    experts = pl.slot_expert
    all_gu, all_d = wgu, wd
    if shared:
        bounds, experts = np.append(bounds, rows), np.append(experts, w.E)
        all_gu, all_d = torch.cat((wgu, sgu)), torch.cat((wd, sd))
    xv = values(x, fmt, layer.x_exp)[src]
    h, err = product(xv, expert_values(all_gu, fmt), bounds, experts, None, w.I)
    near(layer.h[:rows], h, err)
    # down: from the hidden rows that the layer holds
    hv = values(layer.h[:rows], fmt, layer.h_exp)
    yp, err = product(hv, expert_values(all_d, fmt), bounds, experts, None, 0)
    near(layer.y_perm[:rows], yp, err)
    # combine: from the expert rows that the layer holds
    held = layer.y_perm[:rows].float().cpu().numpy().astype(np.float64)
    dest = layer.dest_row[:A].cpu().numpy().reshape(w.T, w.k)
    terms = tw[:, :, None] * held[dest]
    out, mag = terms.sum(1), np.abs(terms).sum(1)
    if shared:
        out, mag = out + held[A:], mag + np.abs(held[A:])
    near(y, out, (w.k + 1) * 2.0 ** -24 * mag)
    # the step as a graph
    y_graph, y_eager = torch.zeros_like(y), torch.zeros_like(y)
    graph = layer.capture(logits, x, y_graph)
    logits.copy_(torch.randn(w.T, w.E, generator=gen, device=dev))
    graph.replay()
    layer.forward(logits, x, y_eager)
    layer.check()
    assert torch.equal(y_graph, y_eager) and not torch.equal(y_eager, y)


def test_router_training_step():
    from grouped_ffn_gb300 import MoELayer
    m = moe()
    w = wl.WORKLOADS["tiny"].scaled(T=64, H=256, I=128, E=32, k=4)
    dev = torch.device("cuda:0")
    pl = wl.make_placement(w)
    logits, x = wl.make_logits(w, dev), wl.make_x(w, dev)
    bias = torch.zeros(w.E, device=dev)
    cfg = m.GateCfg(m.MOE_SCORE_SOFTMAX, w.k, 1, 1, 1, 0, 1.0)
    layer = MoELayer(H=w.H, I=w.I, E=w.E, k=w.k, placement=m.DevicePlacement.from_tables(pl, dev),
                     w_gate_up=wl.make_w_gate_up(w, dev), w_down=wl.make_w_down(w, dev), max_tokens=w.T, device=dev,
                     gate=cfg, gate_bias=bias)
    y = torch.empty(w.T, w.H, dtype=torch.bfloat16, device=dev)
    layer.forward(logits, x, y)
    g = torch.randn(w.T, w.k, device=dev)
    out = torch.empty_like(logits)
    layer.gate_backward(logits, g, out)
    layer.update_gate_bias(0.01)
    layer.check()
    ids = layer.topk_ids.cpu().numpy()
    dl, size = tg.gradient(logits.cpu().numpy().astype(np.float64), ids, g.cpu().numpy().astype(np.float64), 0, 0, 1.0)
    assert (np.abs(out.cpu().numpy() - dl) <= 32 * 2.0 ** -24 * size + 2.0 ** -120).all()
    loads = np.bincount(ids.ravel(), minlength=w.E)
    want = np.float32(0.01) * np.sign(loads.mean() - loads).astype(np.float32)
    assert np.array_equal(layer.gate_bias.cpu().numpy(), want)
    assert layer.gate_bias is bias


def test_refusals():
    from grouped_ffn_gb300 import MoELayer
    m = moe()
    w = wl.WORKLOADS["tiny"]
    dev = torch.device("cuda:0")
    base = dict(H=w.H, I=w.I, E=w.E, k=w.k, placement=m.DevicePlacement.from_tables(wl.make_placement(w), dev),
                w_gate_up=wl.make_w_gate_up(w, dev), w_down=wl.make_w_down(w, dev), max_tokens=w.T, device=dev)
    cfg = m.GateCfg(0, 3, 1, 1, 1, 1, 1.0)
    for bad in (dict(fp4=2), dict(fp4=MX, gather=True), dict(fp4=NV, masked_cap=8), dict(fp4=MX, fp8_dispatch=True),
                dict(gate=cfg), dict(gate_bias=torch.zeros(w.E, device=dev)),
                dict(fp4=MX, shared_w_gate_up=torch.zeros(1, 256, w.H + 256, device=dev))):
        with pytest.raises(ValueError):
            MoELayer(**base, **bad)
