"""Workloads of the router with balance bias, of FP4 rows and of the experts' FP4 product.

Three operators are called here, each in a plain form of elementary torch
operations (own = False) and through the library's entry points (own = True):

  gate      scores of the router's logits, a balance bias, groups, top-k and
            weights (moe_gate); with "train" also the gradient of the logits
            (moe_gate_backward) and the bias update (moe_gate_update_bias)
  rows      rows to 4-bit codes with block scales, into dispatched rows where
            "k" is not 0, and back to values (moe_quantize_fp4 or
            moe_permute_fp4, then moe_dequant_fp4)
  product   bf16 rows in per-expert segments to FP4 and times the experts' FP4
            weights, with SwiGLU where "I" is given
            (moe_quantize_fp4, moe_grouped_product_fp4)
"""

import math
import random

import torch

own = False

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # e2m1 magnitudes
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = {"mx": 32, "nv": 16}


# ------------------------------------------------------------------ cases
def _gate(name, T, E, k, score, groups=1, kept=1, topn=1, bias=True, renorm=True, scale=1.0,
          dtype="f32", masked=0, train=False):
    return dict(name=name, op="gate", T=T, E=E, k=k, score=score, groups=groups, kept=kept,
                topn=topn, bias=bias, renorm=renorm, scale=scale, dtype=dtype, masked=masked,
                train=train)


def _rows(name, T, K, fmt, k=0, dtype="bf16", exp=-8):
    return dict(name=name, op="rows", T=T, K=K, fmt=fmt, k=k, dtype=dtype,
                exp=exp if fmt == "nv" else 0)


def _product(name, rows, E, K, fmt, N=0, I=0, zipf=0.0, out="bf16"):
    return dict(name=name, op="product", rows=rows, E=E, K=K, N=N, I=I, fmt=fmt, zipf=zipf, out=out)


def listed():
    return [
        # one decoding token through a group-limited router of 256 experts
        _gate("gate_token", 1, 256, 8, "sigmoid", 8, 4, 2, scale=2.5),
        # a packed batch of prompts through the same router
        _gate("gate_prompts", 65536, 256, 8, "sigmoid", 8, 4, 2, scale=2.5),
        # a training step of a softmax router whose weights stay unnormalised
        _gate("gate_train_softmax", 16384, 32, 4, "softmax", renorm=False, train=True),
        # a training step with odd sizes, bf16 logits and experts switched off
        _gate("gate_train_odd", 4001, 120, 6, "sigmoid", 6, 3, 2, dtype="bf16", masked=7, train=True),
        # one decoding token's row into eight experts' segments
        _rows("rows_token", 1, 7168, "nv", k=8),
        # a prompt's rows dispatched to eight experts each
        _rows("rows_dispatch", 4096, 7168, "mx", k=8),
        # fp32 rows of an odd shape
        _rows("rows_f32_odd", 1777, 1440, "nv", dtype="f32"),
        # gate/up of the eight experts one token is routed to
        _product("product_token", 8, 64, 7168, "nv", I=2048),
        # gate/up of a decode step: 64 tokens, top-2 of 64 experts
        _product("product_decode", 128, 64, 8192, "mx", I=2048, zipf=1.0),
        # down projection of a prompt: 4096 tokens, top-8 of 256 experts
        _product("product_down", 32768, 256, 2048, "nv", N=7168, zipf=0.8),
        # odd widths, fp32 output
        _product("product_odd", 333, 5, 1440, "mx", N=712, zipf=0.5, out="f32"),
        # a large batch over few experts, bound by the tensor cores
        _product("product_large", 65536, 32, 4096, "nv", I=2048, zipf=0.5),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the same ranges: sizes over their logarithm, odd ones among them."""
    op = rng.choice(("gate", "rows", "product"))
    if op == "gate":
        groups = rng.choice((1, 1, 2, 4, 6, 8))
        per = _log_int(rng, 4, 512 // groups)
        if rng.random() < 0.5:
            per = max(4, per // 4 * 4)
        E = groups * per
        kept = rng.randint((groups + 1) // 2, groups)
        topn = rng.randint(1, min(2, per))
        masked = rng.choice((0, 0, rng.randint(1, max(1, per // 4))))
        k = rng.randint(1, min(8, kept * (per - masked))) if per > masked else 1
        return _gate(None, _log_int(rng, 1, 65536), E, k, rng.choice(("softmax", "sigmoid")),
                     groups, kept, topn, bias=rng.random() < 0.75, renorm=rng.random() < 0.5,
                     scale=rng.choice((1.0, 2.5)), dtype=rng.choice(("f32", "bf16")), masked=masked,
                     train=rng.random() < 0.5)
    if op == "rows":
        fmt = rng.choice(("mx", "nv"))
        k = rng.choice((0, 0, 1, 2, 4, 8))
        dtype = "bf16" if k else rng.choice(("bf16", "f32"))
        K = 32 * _log_int(rng, 4, 256)
        return _rows(None, _log_int(rng, 1, 4096), K, fmt, k=k, dtype=dtype)
    K = 32 * _log_int(rng, 16, 256)
    width = 8 * _log_int(rng, 32, 896)
    swiglu = rng.random() < 0.5
    if swiglu:
        width = max(8, width // 16 * 8)
    n = 2 * width if swiglu else width
    E = min(_log_int(rng, 1, 256), max(1, 256 * 2048 * 7168 // (n * K)))
    rows = min(_log_int(rng, 1, 65536), max(1, 65536 * 4096 * 4096 // (n * K)))
    return _product(None, rows, E, K, rng.choice(("mx", "nv")), N=0 if swiglu else width,
                    I=width if swiglu else 0, zipf=rng.choice((0.0, 0.5, 1.0)),
                    out=rng.choice(("bf16", "bf16", "f32")))


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


def _activations(shape, gen):
    """Unit normal rows whose channels differ in size, as a norm with a learned weight leaves them."""
    channel = torch.exp(0.5 * torch.randn(shape[-1], generator=gen, device="cuda"))
    return torch.randn(shape, generator=gen, device="cuda") * channel


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = random.Random(seed)
    s = dict(case=case)
    if case["op"] == "gate":
        T, E, k = case["T"], case["E"], case["k"]
        # logits of a trained router: unit spread with favoured experts
        logits = torch.randn(T, E, generator=gen, device="cuda")
        logits += 0.5 * torch.randn(E, generator=gen, device="cuda")
        for g in range(case["groups"]):
            per = E // case["groups"]
            for e in rng.sample(range(per), case["masked"]):
                logits[:, g * per + e] = -math.inf
        s["logits"] = logits.to(DTYPES[case["dtype"]])
        s["bias"] = (0.05 * torch.randn(E, generator=gen, device="cuda")) if case["bias"] else None
        s["grad"] = torch.randn(T, k, generator=gen, device="cuda")
        s["counts"] = torch.randint(0, 2 * T * k // E + 2, (E,), generator=gen, device="cuda",
                                    dtype=torch.int32)
        if own:
            from grouped_ffn_gb300 import moe
            s["cfg"] = moe.GateCfg(
                moe.MOE_SCORE_SIGMOID if case["score"] == "sigmoid" else moe.MOE_SCORE_SOFTMAX, k,
                case["groups"], case["kept"], case["topn"], int(case["renorm"]), case["scale"])
            s["ids"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
            s["w"] = torch.empty(T, k, device="cuda")
            s["grad_logits"] = torch.empty_like(s["logits"])
            s["bias_out"] = torch.empty(E, device="cuda")
            s["ws"] = moe.new_workspace(T, k, E)
        return s
    if case["op"] == "rows":
        T, K, k = case["T"], case["K"], case["k"]
        s["x"] = _activations((T, K), gen).to(DTYPES[case["dtype"]])
        n = T * k if k else T
        if k:
            s["dest"] = torch.randperm(n, generator=gen, device="cuda").to(torch.int32)
        if own:
            from grouped_ffn_gb300 import moe
            s["fmt"] = moe.MOE_FP4_NV if case["fmt"] == "nv" else moe.MOE_FP4_MX
            s["codes"], s["sf"] = moe.new_fp4(n, K, s["fmt"])
            s["out"] = torch.empty(n, K, dtype=s["x"].dtype, device="cuda")
            s["ws"] = moe.new_workspace(T, max(k, 1), 1)
        return s
    E, K, rows = case["E"], case["K"], case["rows"]
    N = case["N"] or 2 * case["I"]
    fmt = case["fmt"]
    s["x"] = _activations((rows, K), gen).bfloat16()
    counts = _segments(rows, E, case["zipf"], rng)
    s["bounds"] = [sum(counts[:e]) for e in range(E + 1)]
    x_exp, w_exp = (-8, -14) if fmt == "nv" else (0, 0)
    s["x_exp"] = x_exp
    s["w_codes"] = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
    s["w_scale"] = torch.empty(E, N, K // BLOCK[fmt], device="cuda")
    for e in range(E):
        w = 0.02 * torch.randn(N, K, generator=gen, device="cuda")
        idx, s["w_scale"][e] = _quantize(w.bfloat16().float(), fmt, w_exp)
        s["w_codes"][e] = idx[:, 0::2] + 16 * idx[:, 1::2]
    # one factor an expert: its tensor scale times the rows'
    s["alpha"] = torch.exp(0.2 * torch.randn(E, generator=gen, device="cuda")) * 2.0 ** (x_exp + w_exp)
    if own:
        from grouped_ffn_gb300 import moe
        s["fmt"] = moe.MOE_FP4_NV if fmt == "nv" else moe.MOE_FP4_MX
        s["epilogue"] = moe.MOE_EPI_SWIGLU if case["I"] else moe.MOE_EPI_NONE
        sf = torch.zeros(E, N, moe.moe_fp4_scale_ld(K, s["fmt"]), dtype=torch.uint8, device="cuda")
        if fmt == "nv":
            sf[:, :, :K // 16] = s["w_scale"].to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            sf[:, :, :K // 32] = (torch.frexp(s["w_scale"])[1] + 126).to(torch.uint8)
        s["w"] = moe.pack_weights_fp4(s["w_codes"], sf, s["fmt"], s["epilogue"])
        s["codes"], s["sf"] = moe.new_fp4(rows, K, s["fmt"])
        s["offsets"] = torch.tensor(s["bounds"], dtype=torch.int32, device="cuda")
        s["experts"] = torch.arange(E, dtype=torch.int32, device="cuda")
        s["out"] = torch.empty(rows, case["I"] or N, dtype=DTYPES[case["out"]], device="cuda")
        s["ws"] = moe.new_workspace(rows, 1, E)
    return s


# ------------------------------------------------------------------ plain forms
def _scores(l, score):
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    e = torch.exp(l - l.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _gate_plain(s):
    case, logits = s["case"], s["logits"]
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    # the choice is made in 64 bits: scores next to one another decide it
    off = torch.isneginf(logits)
    c = _scores(logits.double(), case["score"])
    if s["bias"] is not None:
        c = c + s["bias"].double()
    if G > 1:
        best = c.masked_fill(off, -math.inf).view(T, G, E // G).sort(2, descending=True)[0]
        best = best[:, :, :case["topn"]]
        gs = best.masked_fill(torch.isneginf(best), 0).sum(2)
        gs = gs.masked_fill(torch.isneginf(best).all(2), -math.inf)
        order = gs.sort(dim=1, descending=True, stable=True)[1][:, :case["kept"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=c.device).scatter_(1, order, True)
        out = ~keep.repeat_interleave(E // G, 1)
    else:
        out = torch.zeros_like(off)
    c = c.masked_fill(off, -1e300).masked_fill(out, -math.inf)
    ids = c.sort(dim=1, descending=True, stable=True)[1][:, :k]
    sc = _scores(logits.float(), case["score"])
    sel = sc.gather(1, ids)
    w = case["scale"] * sel
    if case["renorm"]:
        w = w / sel.sum(1, keepdim=True)
    res = [ids.to(torch.int32), w]
    if case["train"]:
        g = case["scale"] * s["grad"]
        if case["renorm"]:
            total = sel.sum(1, keepdim=True)
            ds = (g - (g * sel).sum(1, keepdim=True) / total) / total
        else:
            ds = g
        if case["score"] == "sigmoid":
            dl = torch.zeros_like(sc).scatter_(1, ids, ds * sel * (1 - sel))
        else:
            dl = sc * (torch.zeros_like(sc).scatter_(1, ids, ds) - (ds * sel).sum(1, keepdim=True))
        res.append(dl.to(logits.dtype))
        if s["bias"] is not None:
            n = s["counts"].to(torch.int64)
            res.append(s["bias"] + 0.001 * torch.sign(n.sum() - E * n).float())
    return res


def _quantize(x, fmt, exp):
    """fp32 rows [n, K] to code numbers 0..15 (uint8) and block scales (fp32, without 2^exp)."""
    blocks = x.view(*x.shape[:-1], -1, BLOCK[fmt])
    amax = blocks.abs().amax(-1)
    if fmt == "mx":
        m, q = torch.frexp(amax)
        e = (q - 3 + (m > 0.75).to(q.dtype)).clamp(-127, 127)
        scale = torch.ldexp(torch.ones_like(amax), e.masked_fill(amax == 0, -127))
    else:
        # (divided by a tensor: torch multiplies by the reciprocal of a number)
        v = (amax * 2.0 ** -exp / torch.full_like(amax, 6)).clamp(max=448.0)
        step = torch.exp2(torch.floor(torch.log2(v.clamp(min=2.0 ** -6))) - 3)
        scale = (torch.round(v / step) * step).to(x.dtype)
    y = blocks.abs() / (scale * 2.0 ** exp).unsqueeze(-1)
    y = y.masked_fill((scale == 0).unsqueeze(-1), 0)
    idx = torch.zeros(y.shape, dtype=torch.uint8, device=x.device)
    for t in (0.25, 1.25, 2.5, 5.0):   # halfway goes to the even code, below
        idx += y > t
    for t in (0.75, 1.75, 3.5):        # and above
        idx += y >= t
    idx += 8 * (blocks < 0).to(torch.uint8)
    return idx.view(x.shape), scale.float()


def _values(idx, scale, fmt, exp):
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device=idx.device)
    v = grid[idx.to(torch.int64)].view(*idx.shape[:-1], -1, BLOCK[fmt])
    return (v * (scale * 2.0 ** exp).unsqueeze(-1)).view(idx.shape)


def _rows_plain(s):
    case, x = s["case"], s["x"]
    # quotients of fp32 rows next to a border need 64 bits, those of bf16 rows do not
    wide = torch.float64 if case["dtype"] == "f32" else torch.float32
    idx, scale = _quantize(x.to(wide), case["fmt"], case["exp"])
    v = _values(idx, scale, case["fmt"], case["exp"]).to(x.dtype)
    if not case["k"]:
        return v
    out = torch.empty(case["T"] * case["k"], case["K"], dtype=x.dtype, device=x.device)
    out[s["dest"].long()] = v.repeat_interleave(case["k"], 0)
    return out


def _product_plain(s):
    case, b = s["case"], s["bounds"]
    idx, scale = _quantize(s["x"].float(), case["fmt"], s["x_exp"])
    x = _values(idx, scale, case["fmt"], 0)
    out = torch.empty(case["rows"], case["I"] or case["N"], dtype=DTYPES[case["out"]],
                      device=x.device)
    for e in range(case["E"]):
        if b[e] == b[e + 1]:
            continue
        c = s["w_codes"][e]
        w = _values(torch.stack((c % 16, c // 16), -1).view(c.shape[0], -1), s["w_scale"][e],
                    case["fmt"], 0)
        y = (x[b[e]:b[e + 1]] @ w.T) * s["alpha"][e]
        if case["I"]:
            g, u = y[:, :case["I"]], y[:, case["I"]:]
            y = g / (1 + torch.exp(-g)) * u
        out[b[e]:b[e + 1]] = y.to(out.dtype)
    return out


# ------------------------------------------------------------------ one pass
def run(s):
    case = s["case"]
    if not own:
        return {"gate": _gate_plain, "rows": _rows_plain, "product": _product_plain}[case["op"]](s)
    from grouped_ffn_gb300 import moe
    if case["op"] == "gate":
        moe.moe_gate(s["logits"], s["bias"], s["cfg"], s["ids"], s["w"])
        res = [s["ids"], s["w"]]
        if case["train"]:
            moe.moe_gate_backward(s["logits"], s["ids"], s["grad"], s["cfg"], s["grad_logits"],
                                  s["ws"])
            res.append(s["grad_logits"])
            if s["bias"] is not None:
                moe.moe_gate_update_bias(s["counts"], s["bias"], 0.001, s["bias_out"])
                res.append(s["bias_out"])
        return res
    if case["op"] == "rows":
        if case["k"]:
            moe.moe_permute_fp4(s["x"], case["k"], s["dest"], s["fmt"], case["exp"], s["codes"],
                                s["sf"], s["ws"])
        else:
            moe.moe_quantize_fp4(s["x"], s["fmt"], case["exp"], s["codes"], s["sf"])
        moe.moe_dequant_fp4(s["codes"], s["sf"], s["fmt"], case["exp"], s["out"])
        return s["out"]
    moe.moe_quantize_fp4(s["x"], s["fmt"], s["x_exp"], s["codes"], s["sf"])
    moe.moe_grouped_product_fp4(s["codes"], s["sf"], s["offsets"], s["experts"], s["w"], s["alpha"],
                                s["out"], s["ws"])
    return s["out"]


# ------------------------------------------------------------------ work
def work(case):
    if case["op"] == "gate":
        T, E, k = case["T"], case["E"], case["k"]
        b = 4 if case["dtype"] == "f32" else 2
        n = T * E * b + T * k * 8 + (4 * E if case["bias"] else 0)
        if case["train"]:
            n += T * k * 4 + T * E * b + (8 * E if case["bias"] else 0)
        return {"bytes": n, "flops": 10 * T * E}
    if case["op"] == "rows":
        T, K = case["T"], case["K"]
        b = 4 if case["dtype"] == "f32" else 2
        n = T * max(case["k"], 1)
        fp4 = K // 2 + K // BLOCK[case["fmt"]]
        return {"bytes": T * K * b + n * (2 * fp4 + K * b) + (4 * n if case["k"] else 0),
                "flops": 3 * T * K}
    K, rows = case["K"], case["rows"]
    N = case["N"] or 2 * case["I"]
    used = sum(1 for c in _segments(rows, case["E"], case["zipf"], random.Random(0)) if c)
    fp4 = K // 2 + K // BLOCK[case["fmt"]]
    out = (case["I"] or N) * (4 if case["out"] == "f32" else 2)
    return {"bytes": rows * (2 * K + out) + used * N * fp4, "flops": 2 * rows * N * K}


# ------------------------------------------------------------------ 64 bits
def _exact_gate(s):
    case = s["case"]
    l = s["logits"].double()
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    dead = l == -math.inf
    if case["score"] == "sigmoid":
        p = torch.where(l >= 0, 1 / (1 + torch.exp(-l.abs())),
                        torch.exp(-l.abs()) / (1 + torch.exp(-l.abs())))
    else:
        p = torch.exp(l - torch.logsumexp(l, 1, keepdim=True))
    key = p.clone() if s["bias"] is None else p + s["bias"].double()
    key[dead] = -math.inf
    allowed = torch.ones(T, E, dtype=torch.bool, device=l.device)
    if G > 1:
        per = E // G
        kk = key.reshape(T, G, per).clone()
        total = torch.zeros(T, G, dtype=torch.float64, device=l.device)
        some = (kk > -math.inf).any(2)
        for _ in range(case["topn"]):
            v, i = kk.max(2)
            total += torch.where(v > -math.inf, v, 0)
            kk.scatter_(2, i.unsqueeze(2), -math.inf)
        total[~some] = -math.inf
        allowed.zero_()
        for _ in range(case["kept"]):
            # the first of the largest, among the groups not taken yet
            free = torch.isnan(total).logical_not()
            m = torch.where(free, total, -math.inf)
            top = (free & (m == m.amax(1, keepdim=True))).to(torch.uint8).argmax(1, keepdim=True)
            total.scatter_(1, top, math.nan)
            allowed.view(T, G, per).scatter_(1, top.unsqueeze(2).expand(-1, -1, per), True)
    free = allowed
    ids = torch.empty(T, k, dtype=torch.int64, device=l.device)
    for j in range(k):
        m = torch.where(free, key, -math.inf)
        best = free & (m == m.amax(1, keepdim=True))
        i = best.to(torch.uint8).argmax(1, keepdim=True)
        ids[:, j:j + 1] = i
        free = free.scatter(1, i, False)
    ps = p.gather(1, ids)
    z = ps.sum(1, keepdim=True)
    w = case["scale"] * (ps / z if case["renorm"] else ps)
    res = [ids.to(torch.int32), w]
    if case["train"]:
        up = torch.zeros(T, E, dtype=torch.float64, device=l.device)
        up.scatter_(1, ids, s["grad"].double() * case["scale"])
        if case["renorm"]:
            v = ps / z
            mean = (up.gather(1, ids) * v).sum(1, keepdim=True)
            up = torch.zeros_like(up).scatter_(1, ids, (up.gather(1, ids) - mean) / z)
        if case["score"] == "sigmoid":
            q = torch.where(l >= 0, torch.exp(-l.abs()), 1.0) / (1 + torch.exp(-l.abs()))
            dl = up * p * q
        else:
            dl = p * (up - (up * p).sum(1, keepdim=True))
        res.append(dl)
        if s["bias"] is not None:
            n = s["counts"].double()
            res.append(s["bias"].double() + 0.001 * torch.sign(n.mean() - n))
    return res


def _exact_values(x, fmt, exp):
    """The value each element of x (64 bits) is held as, over 2^exp, by nearest grid point."""
    b = x.reshape(-1, BLOCK[fmt])
    top = b.abs().amax(1, keepdim=True)
    if fmt == "mx":
        e = torch.ceil(torch.log2(top / 6)).clamp(-127, 127)
        # settle the rounding of the logarithm
        e = torch.where(top > 6 * torch.exp2(e), e + 1, e)
        e = torch.where((top <= 6 * torch.exp2(e - 1)) & (e > -127), e - 1, e).clamp(-127, 127)
        scale = torch.exp2(e)
    else:
        # the 127 finite e4m3 magnitudes
        code = torch.arange(127, device=x.device)
        mag = torch.where(code < 8, (code % 8) * 2.0 ** -9,
                          (8 + code % 8) * torch.exp2((code // 8).double() - 10))
        scale = _nearest(top * 2.0 ** -exp / torch.full_like(top, 6), mag)
    grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)
    unit = torch.where(scale > 0, scale * 2.0 ** exp, 1.0)
    v = _nearest(b.abs() / unit, grid) * torch.sign(b) * scale
    return v.reshape(x.shape)


def _nearest(v, grid):
    hi = torch.searchsorted(grid, v.contiguous()).clamp(1, len(grid) - 1)
    below, above = v - grid[hi - 1], grid[hi] - v
    even = (hi % 2 == 0)
    return torch.where((above < below) | ((above == below) & even), grid[hi], grid[hi - 1])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "gate":
        return _exact_gate(s)
    if case["op"] == "rows":
        x = s["x"]
        if not case["k"]:
            return _exact_values(x.double(), case["fmt"], case["exp"]) * 2.0 ** case["exp"]
        v = torch.cat([_exact_values(c.double(), case["fmt"], case["exp"]).float()
                       for c in x.split(512)]) * 2.0 ** case["exp"]
        out = torch.empty(case["T"] * case["k"], case["K"], device=x.device)
        for j in range(case["k"]):
            out[s["dest"][j::case["k"]].long()] = v
        return out.double()
    b, fmt = s["bounds"], case["fmt"]
    if case["rows"] * case["K"] * (case["N"] or 2 * case["I"]) > 65536 * 4096 * 4096:
        return None
    grid = torch.tensor(GRID, dtype=torch.float64, device="cuda")
    table = torch.cat((grid, -grid))
    outs = []
    for e in range(case["E"]):
        x = _exact_values(s["x"][b[e]:b[e + 1]].double(), fmt, s["x_exp"]) if b[e + 1] > b[e] else None
        if x is None:
            continue
        c = s["w_codes"][e].int()
        w = torch.empty(c.shape[0], case["K"], dtype=torch.float64, device="cuda")
        w[:, 0::2] = table[(c & 15).long()]
        w[:, 1::2] = table[(c >> 4).long()]
        w *= s["w_scale"][e].double().repeat_interleave(BLOCK[fmt], 1)
        y = torch.matmul(x, w.t()) * s["alpha"][e].double()
        if case["I"]:
            g, u = y.split(case["I"], 1)
            y = g * u / (1 + torch.exp(-g))
        outs.append(y)
    return torch.cat(outs)
