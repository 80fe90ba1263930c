"""The layer inside its block: norm, router, sort, experts (bf16 or 4-bit), weighted
return with norm, gate and residual, as one step, as a graph and as a training step.

Each step is checked against its definition on the step's own inputs, with the
bounds of test_block and test_int4_product.  The training step as a whole is
checked against autograd in 64 bits with the same experts chosen: on the way lie
the roundings to bf16 of n, h, the experts' rows, their gradient, the hidden rows'
two gradients and the dispatched rows' gradient, seven of at most 2^-8 of a value
each, so results are within 7 * 2^-8 in the Frobenius norm (a gradient's terms do
not cancel more than its value, up to the factor of two that the norms add).
"""

import numpy as np
import pytest
import torch

import workloads as wl
from test_block import BF, EPS, F32, Block, Norm, f64, near
from test_int4_product import product


def moe():
    from grouped_ffn_gb300 import moe as m
    return m


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_ffn_gb300 import build
    build.build()


def test_refusals():
    from grouped_ffn_gb300 import MoELayer
    m = moe()
    base = dict(H=256, I=128, E=4, k=2, placement=None, w_gate_up=torch.empty(4, 256, 256), max_tokens=8,
                w_down=torch.empty(4, 256, 128))
    packed = lambda N, K, ep, g=32: m.Int4Weights(torch.empty(0), 4, N, K, g, False, ep)
    gu, dn = packed(256, 256, m.MOE_EPI_SWIGLU), packed(256, 128, m.MOE_EPI_NONE)
    two = dict(w_gate_up=gu, w_down=dn)
    for bad in (dict(int4=16), dict(int4=64, fp4=m.MOE_FP4_MX), dict(int4=64, gather=True), dict(int4=64, masked_cap=4),
                dict(int4=64, fp8_dispatch=True), dict(int4=64, I=96), dict(int4=128, H=320),
                dict(int4=64, shared_w_gate_up=torch.empty(1, 64, 256)), dict(two, int4=64), dict(two, w_down=gu),
                dict(two, shared_w_gate_up=torch.empty(1, 256, 256)), dict(post_weight=torch.ones(256)),
                dict(next_weight=torch.ones(256)), dict(block=m.BlockCfg(0), post_weight=torch.ones(256))):
        with pytest.raises(ValueError):
            MoELayer(**{**base, **bad})


def make(T, H, I, E, k, shared=False, zipf=0.8, **kw):
    from grouped_ffn_gb300 import MoELayer
    m = moe()
    w = wl.WORKLOADS["tiny"].scaled(T=T, H=H, I=I, E=E, k=k, zipf_s=zipf)
    dev = torch.device("cuda:0")
    torch.cuda.set_device(0)
    pl = wl.make_placement(w)
    gen = torch.Generator(device=dev)
    gen.manual_seed(4)
    rn = lambda *s: torch.randn(*s, generator=gen, device=dev)
    d = dict(logits=wl.make_logits(w, dev), x=rn(T, H), pre=1 + 0.2 * rn(H), gate=torch.sigmoid(rn(T)),
             wgu=(0.05 * rn(E, 2 * I, H)).to(BF), wd=(0.05 * rn(E, H, I)).to(BF), pl=pl,
             sgu=(0.05 * rn(1, 2 * I, H)).to(BF) if shared else None,
             sd=(0.05 * rn(1, H, I)).to(BF) if shared else None, rn=rn)
    kw.setdefault("block", m.BlockCfg(1, EPS, 0.5))
    layer = MoELayer(H=H, I=I, E=E, k=k, placement=m.DevicePlacement.from_tables(pl, dev), w_gate_up=d["wgu"],
                     w_down=d["wd"], max_tokens=T + 3, shared_w_gate_up=d["sgu"], shared_w_down=d["sd"], device=dev,
                     post_weight=1 + 0.2 * rn(H), next_weight=1 + 0.2 * rn(H), **kw)
    return layer, d


def int4_values(w, group):
    from grouped_ffn_gb300 import MoELayer
    codes, scales = MoELayer._quantize_int4(w, group)
    q = torch.stack((codes % 16, codes // 16), -1).flatten(2).double() - 8
    v = (q * scales.double().repeat_interleave(group, 2)).cpu().numpy()
    # the nearest of scale * (-7..7): within half a scale, and a bf16 scale's rounding at the ends
    s = scales.double().repeat_interleave(group, 2).cpu().numpy()
    assert (np.abs(v - f64(w)) <= 0.5 * s + 7 * 2.0 ** -8 * s).all()
    return v


def tail_state(layer, d, T, shared, x):
    return dict(dest=layer.dest_row[:T * layer.k].view(T, layer.k), w=layer.topk_w[:T], yp=layer.y_perm,
                shared=shared, x=x, gate=d["gate"], weight=layer.post_weight)


@pytest.mark.gpu
@pytest.mark.parametrize("shared,group", [(False, 128), (True, 32), (True, 64)])
def test_int4_step(shared, group):
    m = moe()
    T, H, I, E, k = 37, 512, 256, 16, 3
    layer, d = make(T, H, I, E, k, shared, int4=group)
    n, y, nx = (torch.empty(T, H, dtype=t, device="cuda") for t in (BF, F32, BF))
    m.moe_norm(d["x"], d["pre"], EPS, n)
    layer.forward(d["logits"], n, y, residual=d["x"], gate=d["gate"], next_out=nx)
    layer.check()
    near(n, *Norm(f64(d["x"])).out(f64(d["pre"])), "n")
    A, rows = T * k, T * k + (T if shared else 0)
    src = layer.src_assign[:A].cpu().numpy() // k
    if shared:
        src = np.concatenate((src, np.arange(T)))
    bounds, experts = layer.seg_offsets.cpu().numpy(), d["pl"].slot_expert
    gu, dn = d["wgu"], d["wd"]
    if shared:
        bounds, experts = np.append(bounds, rows), np.append(experts, E)
        gu, dn = torch.cat((gu, d["sgu"])), torch.cat((dn, d["sd"]))
    near(layer.h[:rows], *product(f64(n)[src], int4_values(gu, group), bounds, experts, I), "h")
    near(layer.y_perm[:rows], *product(f64(layer.h[:rows]), int4_values(dn, group), bounds, experts, 0), "experts")
    st = tail_state(layer, d, T, layer.shared_output(T), d["x"])
    near(y, *Block(st, T, H, True, 0.5).forward(), "y")
    near(nx, *Norm(f64(y)).out(f64(layer.next_weight)), "next")
    # the same step as a graph, in place on the residual, and without a residual
    x2, nx2 = d["x"].clone(), torch.empty_like(nx)
    g = layer.capture(d["logits"], n, x2, residual=x2, gate=d["gate"], next_out=nx2)
    x2.copy_(d["x"])
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(x2, y) and torch.equal(nx2, nx)
    plain = torch.empty(T, H, dtype=BF, device="cuda")
    layer.forward(d["logits"], n, plain)
    layer.check()
    b = Block({**st, "gate": None, "weight": None}, T, H, False, 0.0)
    near(plain, b.c, b.dc, "sum")


@pytest.mark.gpu
def test_packed_int4_weights_are_taken_as_they_are():
    from grouped_ffn_gb300 import MoELayer
    m = moe()
    T, H, I, E, k = 20, 256, 128, 8, 2
    layer, d = make(T, H, I, E, k, int4=64)
    x, y1, y2 = (torch.empty(T, H, dtype=BF, device="cuda") for _ in range(3))
    x.copy_(d["x"])
    layer.forward(d["logits"], x, y1)
    pack = lambda w, ep: m.pack_weights_int4(*MoELayer._quantize_int4(w, 64), None, ep)
    other = MoELayer(H=H, I=I, E=E, k=k, placement=layer.placement, w_gate_up=pack(d["wgu"], m.MOE_EPI_SWIGLU),
                     w_down=pack(d["wd"], m.MOE_EPI_NONE), max_tokens=T, device=torch.device("cuda:0"))
    other.forward(d["logits"], x, y2)
    other.check()
    assert torch.equal(y1, y2)
    with pytest.raises(ValueError):
        other.forward(d["logits"], x, y2, residual=x)
    with pytest.raises(ValueError):
        layer.forward(d["logits"], x, y2, gate=d["gate"])


@pytest.mark.gpu
def test_fixed_capacity_with_a_residual():
    """Dropped assignments add nothing, and get no gradient."""
    m = moe()
    T, H, I, E, k, cap = 60, 256, 128, 8, 2, 12
    layer, d = make(T, H, I, E, k, zipf=1.5, masked_cap=cap)
    n, y = torch.empty(T, H, dtype=BF, device="cuda"), torch.empty(T, H, device="cuda")
    m.moe_norm(d["x"], d["pre"], EPS, n)
    layer.forward(d["logits"], n, y, residual=d["x"], gate=d["gate"])
    layer.check()
    assert layer.n_dropped.item() > 0
    st = tail_state(layer, d, T, None, d["x"])
    near(y, *Block(st, T, H, True, 0.5).forward(), "y")
    gy = d["rn"](T, H)
    rows, gw = torch.full((E * cap, H), 7.0, dtype=BF, device="cuda"), torch.empty(T, k, device="cuda")
    layer.combine_backward(gy, rows, gw, gate=d["gate"])
    layer.check()
    want = Block({**st, "gy": gy}, T, H, True, 0.5).backward()
    near(gw, *want["w"], "w")
    live = st["dest"].cpu().numpy() >= 0
    near(rows[st["dest"][st["dest"] >= 0].long()], want["rows"][0][live], want["rows"][1][live], "rows")
    free = torch.ones(E * cap, dtype=torch.bool)
    free[st["dest"][st["dest"] >= 0].long().cpu()] = False
    assert (rows[free] == 7.0).all()


def experts_backward(rows, grad, bounds, experts, wgu, wd):
    """Gradient of the experts' rows in fp32, each result held in bf16."""
    out = torch.zeros_like(rows)
    I = wd.shape[2]
    for s, e in enumerate(experts):
        lo, hi = int(bounds[s]), int(bounds[s + 1])
        if lo == hi:
            continue
        gu = rows[lo:hi].float() @ wgu[e].float().T
        g, u = gu[:, :I], gu[:, I:]
        sg = torch.sigmoid(g)
        dh = (grad[lo:hi].float() @ wd[e].float()).to(BF).float()
        dgu = torch.cat((dh * u * sg * (1 + g * (1 - sg)), dh * g * sg), 1).to(BF).float()
        out[lo:hi] = (dgu @ wgu[e].float()).to(BF)
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("shared", [False, True])
def test_training_step(shared):
    m = moe()
    T, H, I, E, k = 45, 256, 128, 8, 3
    cfg = m.GateCfg(m.MOE_SCORE_SIGMOID, k, 1, 1, 1, 1, 1.0)
    layer, d = make(T, H, I, E, k, shared, gate=cfg)
    wr = 0.1 * d["rn"](E, H)
    n, y = torch.empty(T, H, dtype=BF, device="cuda"), torch.empty(T, H, device="cuda")
    m.moe_norm(d["x"], d["pre"], EPS, n)
    logits = (n.float() @ wr.T).contiguous()
    layer.forward(logits, n, y, residual=d["x"], gate=d["gate"])
    gy = d["rn"](T, H)
    A, rows = T * k, T * k + (T if shared else 0)
    e = lambda *s, t=F32: torch.empty(*s, dtype=t, device="cuda")
    g_rows, g_w, g_gate, g_post = e(rows, H, t=BF), e(T, k), e(T), e(H)
    layer.combine_backward(gy, g_rows, g_w, gate=d["gate"], grad_shared=g_rows[A:] if shared else None,
                           grad_weight=g_post, grad_gate=g_gate)
    bounds, experts, gu, dn = layer.seg_offsets.cpu().numpy(), d["pl"].slot_expert, d["wgu"], d["wd"]
    if shared:
        bounds, experts = np.append(bounds, rows), np.append(experts, E)
        gu, dn = torch.cat((gu, d["sgu"])), torch.cat((dn, d["sd"]))
    g_in = experts_backward(layer.x_perm[:rows], g_rows, bounds, experts, gu, dn)
    g_logits = e(T, E)
    layer.gate_backward(logits, g_w, g_logits)
    add = g_logits @ wr
    if shared:
        add = add + g_in[A:].float()
    gx, g_pre, g_n = e(T, H), e(H), e(T, H)
    layer.norm_backward(g_in, d["x"], d["pre"], EPS, gx, g_pre, add=add.to(BF), residual_grad=gy)
    layer.permute_backward(g_in, g_n, add=add.to(BF))
    layer.check()

    # autograd in 64 bits, the same experts chosen
    leaf = lambda t: t.double().requires_grad_()
    x, pre, post, gate = leaf(d["x"]), leaf(d["pre"]), leaf(layer.post_weight), leaf(d["gate"])
    norm = lambda v, w: v / torch.sqrt((v * v).mean(1, keepdim=True) + EPS) * w
    nn = norm(x, pre)
    nn.retain_grad()
    ids = layer.topk_ids[:T].long()
    s = torch.sigmoid(nn @ wr.double().T).gather(1, ids)
    w = s / s.sum(1, keepdim=True)
    w.retain_grad()

    def expert(v, i):
        z = v @ gu[i].double().T
        return (z[:, :I] * torch.sigmoid(z[:, :I]) * z[:, I:]) @ dn[i].double().T

    c = expert(nn, E) if shared else torch.zeros_like(nn)
    for i in range(E):
        t, j = (ids == i).nonzero(as_tuple=True)
        if len(t):
            c = c.index_add(0, t, w[t, j].unsqueeze(1) * expert(nn[t], i))
    want = 0.5 * x + gate.unsqueeze(1) * norm(c, post)
    want.backward(gy.double())
    for name, got, ref in (("y", y, want), ("x", gx, x.grad), ("n", g_n, nn.grad), ("pre", g_pre, pre.grad),
                           ("post", g_post, post.grad), ("gate", g_gate, gate.grad), ("w", g_w, w.grad)):
        err = (got.double() - ref.detach()).norm() / ref.detach().norm()
        assert err <= 7 * 2.0 ** -8, (name, err.item())
