"""Workloads of the block around the experts and of its gradient, and of the experts' 4-bit weights.

Three operators are called here, each in a plain form of elementary torch
operations (own = False) and through the library's entry points (own = True):

  sort   gradient of tokens sorted by expert and back: of the weighted sum
         (moe_combine_backward: the experts' rows and the router's weights) and
         of the copies (moe_permute_backward: the tokens)
  block  norms before and after the experts, with the block's gate and its
         residual scale: moe_norm where "pre" is set, moe_combine_norm, which
         also writes the next block's normalised rows where "next" is set; with
         "train" the gradients (moe_combine_norm_backward, moe_norm_backward)
  int4   bf16 rows in per-expert segments times 4-bit weights with group
         scales, with SwiGLU where "I" is given (moe_grouped_product_int4)
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------ cases
def _sort(name, T, H, k, dtype="bf16", drop=0.0, add=True):
    return dict(name=name, op="sort", T=T, H=H, k=k, dtype=dtype, drop=drop, add=add)


def _block(name, T, H, k, dtype="bf16", post=True, gate=False, shared=False, scale=1.0, drop=0.0,
           pre=False, next=False, train=False):
    return dict(name=name, op="block", T=T, H=H, k=k, dtype=dtype, post=post, gate=gate,
                shared=shared, scale=scale, drop=drop, pre=pre, next=next, train=train)


def _int4(name, rows, E, K, group, N=0, I=0, zeros=False, zipf=0.0, out="bf16"):
    return dict(name=name, op="int4", rows=rows, E=E, K=K, N=N, I=I, group=group, zeros=zeros,
                zipf=zipf, out=out)


def listed():
    return [
        # a small training batch's tokens through top-2 of 64 experts
        _sort("sort_small", 64, 8192, 2),
        # a training step on a prompt-sized batch, top-8 of 256 experts
        _sort("sort_train", 4096, 7168, 8),
        # fixed-capacity experts with dropped assignments, fp32 gradients, odd sizes
        _sort("sort_drop_odd", 3001, 1416, 3, dtype="f32", drop=0.15, add=False),
        # one decoding token: after the experts, and the next block's norm
        _block("block_token", 1, 7168, 8, post=False, shared=True, next=True),
        # a decode step with norms on both sides of the experts
        _block("block_decode", 64, 8192, 2, gate=True, next=True),
        # a prompt's tokens, a shared expert beside the routed ones
        _block("block_prompt", 4096, 7168, 8, post=False, shared=True, next=True),
        # a training step with an fp32 residual stream, norms on both sides and a gate
        _block("block_train", 16384, 4096, 4, dtype="f32", gate=True, scale=0.5, pre=True, train=True),
        # a training step of odd sizes with a shared expert and dropped assignments
        _block("block_train_odd", 1777, 1440, 6, shared=True, drop=0.1, pre=True, train=True),
        # gate/up of the eight experts one token is routed to
        _int4("int4_token", 8, 64, 7168, 128, I=2048),
        # gate/up of a decode step: 64 tokens, top-2 of 64 experts
        _int4("int4_decode", 128, 64, 8192, 128, I=2048, zeros=True, zipf=1.0),
        # down projection of a decode step: 64 tokens, top-8 of 256 experts
        _int4("int4_down", 512, 256, 2048, 64, N=7168, zipf=0.8),
        # odd widths, small groups, fp32 output
        _int4("int4_odd", 333, 5, 1440, 32, N=712, zeros=True, zipf=0.5, out="f32"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the same ranges: sizes over their logarithm, odd ones among them."""
    op = rng.choice(("sort", "block", "int4"))
    if op != "int4":
        H = 8 * _log_int(rng, 32, 1024)
        k = rng.randint(2, 8)
        T = min(_log_int(rng, 1, 16384), 16384 * 4096 * 7 // (H * (k + 4)))
        dtype = rng.choice(("bf16", "bf16", "f32"))
        drop = rng.choice((0.0, 0.0, 0.1))
        if op == "sort":
            return _sort(None, T, H, k, dtype, drop, rng.random() < 0.5)
        train = rng.random() < 0.5
        pre = train or rng.random() < 0.3
        post, shared = rng.random() < 0.6, rng.random() < 0.5
        # (the norm of one row alone has hardly a gradient with respect to that row's weight)
        if train and post and not shared:
            drop = 0.0
        return _block(None, T, H, k, dtype, post=post, gate=rng.random() < 0.4,
                      shared=shared, scale=rng.choice((1.0, 0.5, 2.0)), drop=drop,
                      pre=pre, next=not pre, train=train)
    group = rng.choice((32, 64, 128))
    K = group * _log_int(rng, 512 // group, 8192 // group)
    width = 8 * _log_int(rng, 32, 896)
    swiglu = rng.random() < 0.5
    if swiglu:
        width = max(8, width // 16 * 8)
    n = 2 * width if swiglu else width
    E = min(_log_int(rng, 1, 256), max(1, 256 * 2048 * 7168 // (n * K)))
    return _int4(None, _log_int(rng, 1, 512), E, K, group, N=0 if swiglu else width,
                 I=width if swiglu else 0, zeros=rng.random() < 0.5,
                 zipf=rng.choice((0.0, 0.5, 1.0)), out=rng.choice(("bf16", "bf16", "f32")))


# ------------------------------------------------------------------ inputs
def _segments(rows, E, zipf, rng):
    """Rows per expert: Zipf shares in a random expert order, summing to rows."""
    share = [(i + 1) ** -zipf for i in range(E)]
    total = sum(share)
    counts = [int(rows * s / total) for s in share]
    rest = sorted(range(E), key=lambda i: (counts[i] - rows * share[i] / total, i))
    for i in rest[:rows - sum(counts)]:
        counts[i] += 1
    rng.shuffle(counts)
    return counts


def _activations(shape, gen, size=1.0):
    """Rows whose channels differ in size, as a layer with learned weights leaves them."""
    channel = size * torch.exp(0.5 * torch.randn(shape[-1], generator=gen, device="cuda"))
    return torch.randn(shape, generator=gen, device="cuda") * channel


def _dispatch(case, gen):
    """dest_row and the router's weights, renormalised over the chosen experts."""
    T, k = case["T"], case["k"]
    dest = torch.randperm(T * k, generator=gen, device="cuda").to(torch.int32).view(T, k)
    if case["drop"]:
        gone = torch.rand(T, k, generator=gen, device="cuda") < case["drop"]
        gone[:, 0] &= torch.rand(T, generator=gen, device="cuda") < 0.1
        dest = dest.masked_fill(gone, -1)
    w = torch.sigmoid(torch.randn(T, k, generator=gen, device="cuda"))
    return dest.contiguous(), (w / w.sum(1, keepdim=True)).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = random.Random(seed)
    s = dict(case=case)
    if case["op"] == "int4":
        return _prepare_int4(case, s, gen, rng)
    T, H, k = case["T"], case["H"], case["k"]
    A, dt = T * k, DTYPES[case["dtype"]]
    s["dest"], s["w"] = _dispatch(case, gen)
    s["y_perm"] = _activations((A, H), gen, 0.3).bfloat16()
    train = case["op"] == "sort" or case["train"]
    if train:
        s["grad_y"] = (0.1 * torch.randn(T, H, generator=gen, device="cuda")).to(dt)
        s["grad_perm"] = (0.1 * torch.randn(A, H, generator=gen, device="cuda")).bfloat16()
        s["add"] = (0.1 * torch.randn(T, H, generator=gen, device="cuda")).bfloat16()
    if case["op"] == "block":
        s["x"] = _activations((T, H), gen).to(dt)
        s["shared"] = _activations((T, H), gen, 0.3).bfloat16() if case["shared"] else None
        for name in ("pre_weight", "post_weight", "next_weight"):
            s[name] = 1 + 0.2 * torch.randn(H, generator=gen, device="cuda")
        if not case["post"]:
            s["post_weight"] = None
        s["gate"] = torch.sigmoid(torch.randn(T, generator=gen, device="cuda")) if case["gate"] else None
    elif not case["add"]:
        s["add"] = None
    if own:
        from grouped_ffn_gb300 import moe
        s["ws"] = moe.new_workspace(T, k, 1)
        rows = lambda n, t: torch.zeros(n, H, dtype=t, device="cuda")
        if train:
            s["grad_y_perm"] = rows(A, torch.bfloat16)
            s["grad_w"] = torch.empty(T, k, device="cuda")
            s["grad_x"] = rows(T, dt)
        if case["op"] == "block":
            s["cfg"] = moe.BlockCfg(int(case["post"]), EPS, case["scale"])
            s["n"] = rows(T, torch.bfloat16)
            s["y"] = rows(T, dt)
            s["next"] = rows(T, torch.bfloat16) if case["next"] else None
            if train:
                s["scratch"] = moe.new_norm_scratch(T, H)
                s["grad_shared"] = rows(T, torch.bfloat16) if case["shared"] else None
                s["grad_gate"] = torch.empty(T, device="cuda") if case["gate"] else None
                s["grad_post"] = torch.empty(H, device="cuda") if case["post"] else None
                s["grad_pre"] = torch.empty(H, device="cuda")
    return s


def _prepare_int4(case, s, gen, rng):
    E, K, rows, group = case["E"], case["K"], case["rows"], case["group"]
    N = case["N"] or 2 * case["I"]
    s["x"] = _activations((rows, K), gen).bfloat16()
    counts = _segments(rows, E, case["zipf"], rng)
    s["bounds"] = [sum(counts[:e]) for e in range(E + 1)]
    s["codes"] = torch.randint(0, 256, (E, N, K // 2), generator=gen, device="cuda",
                               dtype=torch.uint8)
    s["scales"] = (0.005 * torch.exp(0.3 * torch.randn(E, N, K // group, generator=gen,
                                                       device="cuda"))).bfloat16()
    s["zeros"] = torch.randint(5, 11, (E, N, K // group), generator=gen, device="cuda",
                               dtype=torch.uint8) if case["zeros"] else None
    if own:
        from grouped_ffn_gb300 import moe
        s["weights"] = moe.pack_weights_int4(
            s["codes"], s["scales"], s["zeros"],
            moe.MOE_EPI_SWIGLU if case["I"] else moe.MOE_EPI_NONE)
        s["offsets"] = torch.tensor(s["bounds"], dtype=torch.int32, device="cuda")
        s["experts"] = torch.arange(E, dtype=torch.int32, device="cuda")
        s["out"] = torch.empty(rows, case["I"] or N, dtype=DTYPES[case["out"]], device="cuda")
        s["ws"] = moe.new_workspace(rows, 1, E)
    return s


# ------------------------------------------------------------------ plain forms
def _take(rows, dest):
    """fp32 rows [T, k, H] of an assignment each; zeros for a dropped one."""
    v = rows.float()[dest.clamp(min=0).long()]
    return v.masked_fill((dest < 0).unsqueeze(-1), 0)


def _put(v, dest, like):
    """Assignments' rows [T, k, H] to their places; rows of none stay zero."""
    out = torch.zeros_like(like)
    live = dest >= 0
    out[dest[live].long()] = v[live].to(like.dtype)
    return out


def _sort_plain(s):
    dest, w = s["dest"], s["w"]
    gy = s["grad_y"].float().unsqueeze(1)
    grad_w = (gy * _take(s["y_perm"], dest)).sum(2)
    grad_rows = _put(w.unsqueeze(-1) * gy, dest, s["y_perm"])
    grad_x = _take(s["grad_perm"], dest).sum(1)
    if s["add"] is not None:
        grad_x = grad_x + s["add"].float()
    return [grad_rows, grad_w, grad_x.to(s["grad_y"].dtype)]


def _rstd(x):
    return 1 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)


def _block_plain(s):
    case, dest, w, x = s["case"], s["dest"], s["w"], s["x"].float()
    res = []
    if case["pre"]:
        r = _rstd(x)
        res.append((x * r * s["pre_weight"]).bfloat16())
    rows = _take(s["y_perm"], dest)
    c = (w.unsqueeze(-1) * rows).sum(1)
    if case["shared"]:
        c = c + s["shared"].float()
    g = 1.0 if s["gate"] is None else s["gate"].unsqueeze(1)
    rc, wp = (_rstd(c), s["post_weight"]) if case["post"] else (1.0, 1.0)
    y = (case["scale"] * x + g * (c * rc * wp)).to(s["x"].dtype)
    res.append(y)
    if case["next"]:
        res.append((y.float() * _rstd(y.float()) * s["next_weight"]).bfloat16())
    if not case["train"]:
        return res
    # after the experts
    gy = s["grad_y"].float()
    e = gy * wp
    if case["post"]:
        hat = c * rc
        dc = g * rc * (e - hat * (e * hat).mean(1, keepdim=True))
    else:
        hat, dc = c, g * e
    res += [_put(w.unsqueeze(-1) * dc.unsqueeze(1), dest, s["y_perm"]),
            (dc.unsqueeze(1) * rows).sum(2)]
    if case["shared"]:
        res.append(dc.bfloat16())
    if case["post"]:
        res.append((g * gy * hat).sum(0))
    if s["gate"] is not None:
        res.append((e * hat).sum(1))
    # before the experts
    u = _take(s["grad_perm"], dest).sum(1) + s["add"].float()
    hat = x * r
    e = u * s["pre_weight"]
    dx = case["scale"] * gy + r * (e - hat * (e * hat).mean(1, keepdim=True))
    return res + [dx.to(s["x"].dtype), (u * hat).sum(0)]


def _int4_plain(s):
    case, b = s["case"], s["bounds"]
    out = torch.empty(case["rows"], case["I"] or case["N"], dtype=DTYPES[case["out"]],
                      device=s["x"].device)
    x = s["x"].float()
    for e in range(case["E"]):
        if b[e] == b[e + 1]:
            continue
        c = s["codes"][e]
        q = torch.stack((c % 16, c // 16), -1).float().view(c.shape[0], -1, case["group"])
        z = 8.0 if s["zeros"] is None else s["zeros"][e].float().unsqueeze(-1)
        w = ((q - z) * s["scales"][e].float().unsqueeze(-1)).view(c.shape[0], -1)
        y = x[b[e]:b[e + 1]] @ w.T
        if case["I"]:
            g, u = y[:, :case["I"]], y[:, case["I"]:]
            y = g / (1 + torch.exp(-g)) * u
        out[b[e]:b[e + 1]] = y.to(out.dtype)
    return out


# ------------------------------------------------------------------ one pass
def run(s):
    case = s["case"]
    if not own:
        return {"sort": _sort_plain, "block": _block_plain, "int4": _int4_plain}[case["op"]](s)
    from grouped_ffn_gb300 import moe
    if case["op"] == "int4":
        moe.moe_grouped_product_int4(s["x"], s["offsets"], s["experts"], s["weights"], s["out"],
                                     s["ws"])
        return s["out"]
    if case["op"] == "sort":
        moe.moe_combine_backward(s["grad_y"], s["y_perm"], s["dest"], s["w"], s["grad_y_perm"],
                                 s["grad_w"], s["ws"])
        moe.moe_permute_backward(s["grad_perm"], s["dest"], s["grad_x"], s["ws"], add=s["add"])
        return [s["grad_y_perm"], s["grad_w"], s["grad_x"]]
    res = []
    if case["pre"]:
        moe.moe_norm(s["x"], s["pre_weight"], EPS, s["n"])
        res.append(s["n"])
    moe.moe_combine_norm(s["y_perm"], s["dest"], s["w"], s["x"], s["cfg"], s["y"], s["ws"],
                         shared=s["shared"], weight=s["post_weight"], gate=s["gate"],
                         next_weight=s["next_weight"] if case["next"] else None,
                         next_out=s["next"])
    res.append(s["y"])
    if case["next"]:
        res.append(s["next"])
    if not case["train"]:
        return res
    moe.moe_combine_norm_backward(
        s["grad_y"], s["y_perm"], s["dest"], s["w"], s["cfg"], s["grad_y_perm"], s["grad_w"],
        s["ws"], s["scratch"], shared=s["shared"], weight=s["post_weight"], gate=s["gate"],
        grad_shared=s["grad_shared"], grad_weight=s["grad_post"], grad_gate=s["grad_gate"])
    moe.moe_norm_backward(s["grad_perm"], s["x"], s["pre_weight"], EPS, s["grad_x"], s["grad_pre"],
                          s["ws"], s["scratch"], dest_row=s["dest"], add=s["add"],
                          residual_grad=s["grad_y"], residual_scale=case["scale"])
    res += [s["grad_y_perm"], s["grad_w"]]
    res += [s[n] for n in ("grad_shared", "grad_post", "grad_gate") if s[n] is not None]
    return res + [s["grad_x"], s["grad_pre"]]


# ------------------------------------------------------------------ work
def work(case):
    if case["op"] == "int4":
        K, rows, group = case["K"], case["rows"], case["group"]
        N = case["N"] or 2 * case["I"]
        used = sum(1 for c in _segments(rows, case["E"], case["zipf"], random.Random(0)) if c)
        weights = K // 2 + K // group * (3 if case["zeros"] else 2)
        out = (case["I"] or N) * (4 if case["out"] == "f32" else 2)
        return {"bytes": rows * (2 * K + out) + used * N * weights, "flops": 2 * rows * N * K}
    T, H, k = case["T"], case["H"], case["k"]
    b = 4 if case["dtype"] == "f32" else 2
    # an assignment's rows that are read or written; the first of a token is dropped ten times
    # more rarely
    live = T * (k - case["drop"] * (k - 0.9))
    if case["op"] == "sort":
        # rows, their gradient and the copies' gradient; the token's gradients
        n = 6 * live * H + T * H * (2 * b + (2 if case["add"] else 0)) + 12 * T * k
        return {"bytes": int(n), "flops": int(5 * live * H)}
    n = live * H * 2 + T * H * (2 * b + 2 * (case["pre"] + case["next"] + case["shared"])) + 8 * T * k
    flops = live * H * 2 + 8 * T * H
    if case["train"]:
        n += 4 * live * H + T * H * (2 * b + 2 + 2 * case["shared"]) + 4 * T * k
        flops += 8 * live * H + 20 * T * H
    return {"bytes": int(n), "flops": int(flops)}


# ------------------------------------------------------------------ 64 bits
def _exact_rows(s, name, dest):
    """Leaf rows in 64 bits, and the [T, k, H] that the assignments take from them."""
    leaf = s[name].double().requires_grad_()
    padded = torch.cat((leaf, leaf.new_zeros(1, leaf.shape[1])))
    idx = torch.where(dest >= 0, dest, leaf.shape[0]).long()
    return leaf, torch.index_select(padded, 0, idx.flatten()).unflatten(0, dest.shape)


def _exact_norm(x, weight):
    return x * torch.rsqrt(torch.linalg.vector_norm(x, dim=1, keepdim=True).square() / x.shape[1]
                           + EPS) * weight


def _exact_copies(s, x):
    """Contracts the gradients of the k copies of x with x: its derivative is their sum."""
    dest = s["dest"]
    total = torch.zeros_like(x)
    for j in range(dest.shape[1]):
        t = (dest[:, j] >= 0).nonzero().squeeze(1)
        total = total.index_add(0, t, s["grad_perm"][dest[t, j].long()].double())
    if s["add"] is not None:
        total = total + s["add"].double()
    return (total * x).sum()


def _exact_sort(s):
    leaf, rows = _exact_rows(s, "y_perm", s["dest"])
    w = s["w"].double().requires_grad_()
    y = torch.einsum("tk,tkh->th", w, rows)
    grad_rows, grad_w = torch.autograd.grad(y, (leaf, w), s["grad_y"].double())
    x = torch.zeros(s["grad_y"].shape, dtype=torch.float64, device="cuda", requires_grad=True)
    return [grad_rows, grad_w, torch.autograd.grad(_exact_copies(s, x), x)[0]]


def _exact_block(s):
    case = s["case"]
    x = s["x"].double().requires_grad_()
    leaf, rows = _exact_rows(s, "y_perm", s["dest"])
    w = s["w"].double().requires_grad_()
    leaves = [leaf, w]
    f = torch.einsum("tk,tkh->th", w, rows)
    if case["shared"]:
        leaves.append(s["shared"].double().requires_grad_())
        f = f + leaves[-1]
    if case["post"]:
        leaves.append(s["post_weight"].double().requires_grad_())
        f = _exact_norm(f, leaves[-1])
    if case["gate"]:
        leaves.append(s["gate"].double().requires_grad_())
        f = leaves[-1].unsqueeze(1) * f
    y = case["scale"] * x + f
    pre = s["pre_weight"].double().requires_grad_()
    n = _exact_norm(x, pre)
    res = [n.detach()] if case["pre"] else []
    res.append(y.detach())
    if case["next"]:
        # the next block reads y as it is held
        res.append(_exact_norm(y.detach().to(s["x"].dtype).double(), s["next_weight"].double()))
    if case["train"]:
        res += torch.autograd.grad(y, leaves, s["grad_y"].double(), retain_graph=True)
        down = (y * s["grad_y"].double()).sum() + _exact_copies(s, n)
        res += torch.autograd.grad(down, (x, pre))
    return res


def _exact_int4(s):
    case, b, group = s["case"], s["bounds"], s["case"]["group"]
    out = torch.empty(case["rows"], case["I"] or case["N"], dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        if b[e + 1] == b[e]:
            continue
        c = s["codes"][e].int()
        q = torch.empty(c.shape[0], case["K"], dtype=torch.float64, device="cuda")
        q[:, 0::2] = (c & 15).double()
        q[:, 1::2] = (c >> 4).double()
        q -= 8 if s["zeros"] is None else s["zeros"][e].double().repeat_interleave(group, 1)
        q *= s["scales"][e].double().repeat_interleave(group, 1)
        y = torch.matmul(s["x"][b[e]:b[e + 1]].double(), q.t())
        if case["I"]:
            g, u = y.split(case["I"], 1)
            y = g * torch.sigmoid(g) * u
        out[b[e]:b[e + 1]] = y
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"sort": _exact_sort, "block": _exact_block, "int4": _exact_int4}[case["op"]](s)
