"""The layer with FP4 experts on shapes where its parts meet: a shared
expert's rows behind an odd number of dispatched rows, with widths of an odd
number of 256-element steps; replicas, row tiles of either size and a stream
of the caller; a step without tokens.

Each step of forward is compared with its definition on the step's own inputs
as in test_fp4_layer, with its tolerances.
"""

import numpy as np
import pytest
import torch

import workloads as wl
from test_fp4_layer import expert_values, moe, near, values
from test_fp4_product import product
from test_fp4_rows import MX, NV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_ffn_gb300 import build
    build.build()
    torch.cuda.set_device(0)


def weights(w, shared, seed, dev):
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    rnd = lambda *s: (0.05 * torch.randn(*s, generator=gen, device=dev)).bfloat16()
    one = (rnd(1, 2 * w.I, w.H), rnd(1, w.H, w.I)) if shared else (None, None)
    return rnd(w.E, 2 * w.I, w.H), rnd(w.E, w.H, w.I), *one


def check_step(layer, pl, x, y, wgu, wd, sgu, sd):
    """The layer's buffers after forward(.., x, y) against the definition."""
    T, k, fmt = x.shape[0], layer.k, layer.fp4
    A, shared = T * k, sgu is not None
    rows = A + (T if shared else 0)
    src = layer.src_assign[:A].cpu().numpy() // k
    bounds, experts = layer.seg_offsets.cpu().numpy(), pl.slot_expert
    assert bounds[0] == 0 and bounds[-1] == A
    if shared:
        src = np.concatenate((src, np.arange(T)))
        bounds, experts = np.append(bounds, rows), np.append(experts, layer.E)
        wgu, wd = torch.cat((wgu, sgu)), torch.cat((wd, sd))
    xv = values(x, fmt, layer.x_exp)[src]
    h, err = product(xv, expert_values(wgu, fmt), bounds, experts, None, layer.I)
    near(layer.h[:rows], h, err)
    hv = values(layer.h[:rows], fmt, layer.h_exp)
    yp, err = product(hv, expert_values(wd, fmt), bounds, experts, None, 0)
    near(layer.y_perm[:rows], yp, err)
    held = layer.y_perm[:rows].float().cpu().numpy().astype(np.float64)
    tw = layer.topk_w[:T].cpu().numpy().astype(np.float64)
    terms = tw[:, :, None] * held[layer.dest_row[:A].cpu().numpy().reshape(T, k)]
    out, mag = terms.sum(1), np.abs(terms).sum(1)
    if shared:
        out, mag = out + held[A:], mag + np.abs(held[A:])
    near(y, out, (k + 1) * 2.0 ** -24 * mag)


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("T,k,H,I", [(37, 3, 256, 160), (1, 1, 768, 96), (5, 1, 1280, 288), (9, 3, 768, 64),
                                     (6, 3, 256, 96)])
def test_shared_expert_behind_an_odd_number_of_rows(T, k, H, I, fmt):
    from grouped_ffn_gb300 import MoELayer
    w = wl.WORKLOADS["tiny"].scaled(T=T, H=H, I=I, E=16, k=k)
    dev = torch.device("cuda:0")
    pl = wl.make_placement(w)
    logits, x = wl.make_logits(w, dev), wl.make_x(w, dev)
    ws = weights(w, True, 6, dev)
    layer = MoELayer(H=H, I=I, E=w.E, k=k, placement=moe().DevicePlacement.from_tables(pl, dev), w_gate_up=ws[0],
                     w_down=ws[1], max_tokens=T + 4, shared_w_gate_up=ws[2], shared_w_down=ws[3], device=dev, fp4=fmt)
    for n in (T, T // 2):                       # the layer's largest step, and another
        y = torch.empty(n, H, dtype=torch.bfloat16, device=dev)
        if n == 0:
            continue
        layer.forward(logits[:n].contiguous(), x[:n].contiguous(), y)
        layer.check()
        check_step(layer, pl, x[:n], y, *ws)


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("relax", [None, (5, 4)])
def test_replicas_on_a_stream_of_the_caller(relax, shared, fmt):
    """Experts with replicas, segments long enough for the product's larger row tiles, and steps on a
    stream of the caller whose inputs another stream is still writing."""
    from grouped_ffn_gb300 import MoELayer
    w = wl.WORKLOADS["replica"].scaled(T=901, H=288, I=96, E=32, k=3)
    dev = torch.device("cuda:0")
    pl = wl.make_placement(w)
    logits, x = wl.make_logits(w, dev), wl.make_x(w, dev)
    ws = weights(w, shared, 7, dev)
    layer = MoELayer(H=w.H, I=w.I, E=w.E, k=w.k, placement=moe().DevicePlacement.from_tables(pl, dev), w_gate_up=ws[0],
                     w_down=ws[1], max_tokens=w.T, shared_w_gate_up=ws[2], shared_w_down=ws[3], device=dev, fp4=fmt,
                     replica_relax=relax)
    assert pl.n_slots > w.E and w.T * w.k > 64 * (pl.n_slots + 1)
    late_x, late_logits = torch.zeros_like(x), torch.zeros_like(logits)
    y, ready, side = torch.empty_like(x), torch.cuda.Event(), torch.cuda.Stream()
    layer.forward(logits, x, torch.empty_like(x))
    torch.cuda.synchronize()
    layer._seg_offsets_all.zero_(), layer.h.zero_(), layer.y_perm.zero_()
    busy = torch.randn(8192, 8192, device=dev)
    for _ in range(3):
        busy = busy @ busy * 1e-4
    late_x.copy_(x), late_logits.copy_(logits)
    ready.record()
    side.wait_event(ready)
    layer.forward(late_logits, late_x, y, side)
    side.synchronize()
    layer.check(side)
    check_step(layer, pl, x, y, *ws)


def test_empty_step():
    """No tokens at all: nothing is written, nothing fails."""
    from grouped_ffn_gb300 import MoELayer
    w = wl.WORKLOADS["tiny"].scaled(T=5, H=256, I=96, E=16, k=2)
    dev = torch.device("cuda:0")
    pl = wl.make_placement(w)
    logits, x = wl.make_logits(w, dev), wl.make_x(w, dev)
    ws = weights(w, True, 8, dev)
    layer = MoELayer(H=w.H, I=w.I, E=w.E, k=w.k, placement=moe().DevicePlacement.from_tables(pl, dev), w_gate_up=ws[0],
                     w_down=ws[1], max_tokens=w.T, shared_w_gate_up=ws[2], shared_w_down=ws[3], device=dev, fp4=MX)
    for n in (w.T, 0, w.T):
        y = torch.empty(n, w.H, dtype=torch.bfloat16, device=dev)
        layer.forward(logits[:n], x[:n], y)
        layer.check()
    check_step(layer, pl, x, y, *ws)
