"""A training step's remaining operators as timed workloads: the gated
feed-forward projections and the token log probabilities of hidden states
(without their logits), each with its gradient, and AdamW over many tensors.

`run` computes a case either in plain torch operations (own = False) or with
the library's kernels (own = True); `exact` gives the same outputs in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}
# a drawn case costs at most what the largest listed one of its operator does
GATED_MOST, GATED_GRAD_MOST = 8192 * 16384 * 4096, 8192 * 8192 * 4096
HEAD_MOST, HEAD_GRAD_MOST, LOGITS_MOST = 4096 * 50021 * 4096, 4096 * 131072 * 2048, 4096 * 131072
ADAMW_MOST = 1 << 28
LR, BETA1, BETA2, ADAM_EPS, DECAY, STEP = 1e-3, 0.9, 0.95, 1e-8, 0.1, 1000
GROUP = 256  # values that share a scale of the 8-bit states


def listed():
    return [
        # one token through the gated projections while serving: the weights are read once
        dict(name="gated token", op="gated", M=1, N=16384, K=4096, pad=0, type="bf16", out="bf16", act="silu",
             bias=False, pre=False),
        # a training batch, the two projections kept for the backward pass
        dict(name="gated up", op="gated", M=8192, N=16384, K=4096, pad=0, type="bf16", out="bf16", act="gelu_tanh",
             bias=True, pre=True),
        # a prompt over decoded e4m3 weights, to the e4m3 bytes that the coders take
        dict(name="gated e4m3", op="gated", M=2048, N=16384, K=4096, pad=0, type="e4m3", out="e4m3", act="gelu",
             bias=False, pre=False),
        # a training batch's backward pass
        dict(name="gated grad", op="gated_grad", M=8192, N=8192, K=4096, pad=0, type="bf16", act="silu"),
        # a small layer on a ragged batch, rows that start anywhere
        dict(name="gated grad ragged", op="gated_grad", M=257, N=1000, K=771, pad=0, type="f16", act="gelu"),
        # a decode step's tokens scored by the head, no logits kept
        dict(name="head step", op="head", M=8, V=131072, K=4096, pad=0, type="bf16", scale=1.0),
        # scoring a text under a vocabulary of odd size
        dict(name="head score", op="head", M=4096, V=50021, K=4096, pad=0, type="bf16", scale=0.7),
        # the loss gradient of a training batch, with respect to hidden states and head
        dict(name="head grad", op="head_grad", M=4096, V=131072, K=2048, pad=0, type="bf16", scale=1.0),
        # a small head on a ragged batch
        dict(name="head grad ragged", op="head_grad", M=333, V=8001, K=515, pad=5, type="f16", scale=1.4),
        # the coded feed-forward example's block and head, bf16 weights and float32 norms: latency
        dict(name="adamw block", op="adamw", width=512, hidden=2048, vocab=8000, layers=1, type="bf16", grad="bf16",
             bits=32, master=False, align=GROUP),
        # a model's matrices with their states in 8 bits
        dict(name="adamw 8 bit", op="adamw", width=4096, hidden=16384, vocab=32000, layers=1, type="bf16",
             grad="bf16", bits=8, master=False, align=GROUP),
        # mixed precision: float32 masters and gradients summed in float32
        dict(name="adamw master", op="adamw", width=2048, hidden=8192, vocab=50021, layers=2, type="bf16",
             grad="f32", bits=32, master=True, align=GROUP),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]: odd, a multiple of 8 or of 64."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    kind = rng.randrange(3)
    v = v | 1 if kind == 0 else v // 8 * 8 if kind == 1 else v // 64 * 64
    return min(hi, max(lo, v))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_grad", "head", "head_grad", "adamw", "adamw"])
    pad = rng.choice([0, 0, 8, 5])
    if op in ("gated", "gated_grad"):
        most = GATED_MOST if op == "gated" else GATED_GRAD_MOST
        N, K = _log(rng, 64, 16384), _log(rng, 64, 16384)
        c = dict(op=op, M=_log(rng, 1, max(1, min(8192, most // (N * K)))), N=N, K=K, pad=pad,
                 type=rng.choice(["bf16", "f16"] if op == "gated_grad" else ["bf16", "f16", "e4m3"]),
                 act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]))
        if op == "gated":
            c.update(bias=rng.random() < 0.5, pre=rng.random() < 0.3)
            c["out"] = rng.choice(["bf16", "e4m3"] if c["type"] == "e4m3" else [c["type"], c["type"], "f32"])
        return c
    if op in ("head", "head_grad"):
        V, K = _log(rng, 1000, 262144), _log(rng, 64, 8192)
        most = min(LOGITS_MOST // V, (HEAD_MOST if op == "head" else HEAD_GRAD_MOST) // (V * K))
        return dict(op=op, M=_log(rng, 1, max(1, min(8192, most))), V=V, K=K, pad=pad,
                    type=rng.choice(["bf16", "f16", "e4m3"] if op == "head" else ["bf16", "f16"]),
                    scale=rng.choice([1.0, 0.7, 1.4]))
    total, count = _log(rng, 1000, ADAMW_MOST), _log(rng, 1, 200)
    return dict(op=op, sizes=rng.randrange(1 << 30), count=count, total=total, type=rng.choice(["bf16", "f16", "f32"]),
                grad=rng.choice(["bf16", "f32"]), bits=rng.choice([8, 32]), master=rng.random() < 0.4,
                align=rng.choice([GROUP, GROUP, 8, 1]))


def _shapes(case):
    """[(shape, whether a vector of the norms or biases)] of an update's tensors."""
    if "sizes" in case:  # shares of the total, spread over a factor of a thousand
        rng = random.Random(case["sizes"])
        share = [math.exp(rng.uniform(0, math.log(1000))) for _ in range(case["count"])]
        return [((max(1, int(case["total"] * s / sum(share))),), False) for s in share]
    w, h = case["width"], case["hidden"]
    layer = [((w,), True), ((w,), True), ((h, w), False), ((h,), True), ((w, h), False), ((w,), True)]
    return layer * case["layers"] + [((case["vocab"], w), False)]


def _layout(case):
    """Each tensor's (shape, type, gradient's type, place, length, place and number of its scales): an update's
    tensors lie in one buffer for each type, each on a multiple of case["align"] elements."""
    rows, lo, at = [], 0, 0
    for shape, vector in _shapes(case):
        n = math.prod(shape)
        pt = torch.float32 if vector else TYPES[case["type"]]
        gt = pt if vector else TYPES[case["grad"]]
        groups = (n + GROUP - 1) // GROUP
        rows.append((shape, pt, gt, lo, n, at, groups))
        lo, at = lo + (n + case["align"] - 1) // case["align"] * case["align"], at + groups
    return rows


def _length(case, kind):
    last = _layout(case)[-1]
    return last[5] + last[6] if kind.endswith("scale") else last[3] + last[4]


# ------------------------------------------------------------------ inputs

def _normal(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(dtype)


def _rows(g, rows, cols, pad, dtype, std=1.0):
    """[rows, cols] values in rows of cols + pad elements."""
    t = _normal(g, rows, cols + pad, std=std)
    if dtype == torch.float8_e4m3fn:
        t = t.clamp(-448, 448)
    return t.to(dtype)[:, :cols]


def _products(g, M, N, K, pad, dt, many):
    """x [M, K], `many` weights [N, K] and the scale that makes their product's variance 1."""
    x = _rows(g, M, K, pad, dt)
    if dt == torch.float8_e4m3fn:  # weights in units of their scale
        return x, [_rows(g, N, K, pad, dt, std=16.0) for _ in range(many)], 1 / (16.0 * math.sqrt(K))
    return x, [_rows(g, N, K, pad, dt, std=1 / math.sqrt(K)) for _ in range(many)], 1.0


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op = case["op"]
    s = dict(case=case)
    if op == "adamw":
        for i, (shape, pt, gt, lo, n, at, groups) in enumerate(_layout(case)):
            size = 10.0 ** float(torch.rand((), generator=g, device=DEV) * 2 - 4)  # this tensor's gradients
            p = _normal(g, n, std=0.02)
            parts = {"param": (pt, lo, p), "grad": (gt, lo, _normal(g, n, std=size))}
            if case["bits"] == 8:
                parts.update(m=(torch.float8_e4m3fn, lo, _normal(g, n, std=100.0).clamp(-448, 448)),
                             v=(torch.float8_e4m3fn, lo, (_normal(g, n, std=0.5) + 4).exp().clamp(1, 448)),
                             m_scale=(torch.float32, at, _normal(g, groups, std=0.3).exp() * (size * 0.002)),
                             v_scale=(torch.float32, at, _normal(g, groups, std=0.3).exp() * (size * 0.02)))
            else:
                parts.update(m=(torch.float32, lo, _normal(g, n, std=size * 0.25)),
                             v=(torch.float32, lo, (_normal(g, n, std=0.5).exp() * size).square()))
            if case["master"] and pt != torch.float32:
                parts["master"] = (torch.float32, lo, p)
            for k, (dt, first, values) in parts.items():
                flat = s.setdefault("flat", {}).get((k, dt))
                if flat is None:
                    flat = s["flat"][k, dt] = torch.zeros(_length(case, k), dtype=dt, device=DEV)
                view = flat[first:first + values.numel()]
                view.copy_(values)
                s.setdefault(k, {})[i] = view if k.endswith("scale") else view.view(shape)
        return s
    M, K, pad, dt = case["M"], case["K"], case["pad"], TYPES[case["type"]]
    if op in ("gated", "gated_grad"):
        N = case["N"]
        x, (wg, wu), s["scale"] = _products(g, M, N, K, pad, dt, 2)
        s.update(x=x, w_gate=wg, w_up=wu, up_scale=s["scale"] * (0.75 if dt.itemsize == 1 else 1.0))
        if op == "gated":
            bt = torch.bfloat16 if dt.itemsize == 1 else dt
            b = [_normal(g, N, std=0.5, dtype=bt) if case["bias"] else None for _ in range(2)]
            s.update(bias_gate=b[0], bias_up=b[1], out_scale=16.0)
        else:
            s.update(dy=_rows(g, M, N, pad, dt, std=0.1), pre_gate=_rows(g, M, N, pad, dt),
                     pre_up=_rows(g, M, N, pad, dt))
        return s
    V = case["V"]
    x, (w,), unit = _products(g, M, V, K, pad, dt, 1)
    tok = torch.randint(0, V, (M,), generator=g, device=DEV)
    tok[torch.rand(M, generator=g, device=DEV) < 0.05] = -1  # positions without a token
    s.update(x=x, w=w, tokens=tok, scale=case["scale"] * 2.5 * unit)
    if op == "head_grad":
        lse, ent = [], []
        step = max(1, (1 << 28) // V)
        for i in range(0, M, step):
            z = (x[i:i + step].float() @ w.float().T) * s["scale"]
            one = torch.logsumexp(z, -1)
            lse.append(one)
            ent.append(one - (torch.softmax(z, -1) * z).sum(-1))
        s.update(lse=torch.cat(lse), entropy=torch.cat(ent), dlogprob=-(torch.rand(M, generator=g, device=DEV) + 0.5),
                 dentropy=_normal(g, M, std=0.1))
    return s


# ------------------------------------------------------------------ the operators in plain form

def _act(kind, a):
    if kind == "none":
        return a
    if kind == "relu":
        return torch.where(a > 0, a, 0)
    if kind == "gelu":
        return 0.5 * a * (1 + torch.erf(a * math.sqrt(0.5)))
    if kind == "gelu_tanh":
        return 0.5 * a * (1 + torch.tanh(math.sqrt(2 / math.pi) * (a + 0.044715 * a * a * a)))
    return a * torch.sigmoid(a)


def _act_slope(kind, a):
    if kind == "none":
        return torch.ones_like(a)
    if kind == "relu":
        return (a > 0).to(a.dtype)
    if kind == "gelu":
        return 0.5 * (1 + torch.erf(a * math.sqrt(0.5))) + a * torch.exp(-0.5 * a * a) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (a + 0.044715 * a * a * a))
        return 0.5 * (1 + t) + 0.5 * a * (1 - t * t) * c * (1 + 3 * 0.044715 * a * a)
    s = torch.sigmoid(a)
    return s * (1 + a * (1 - s))


def _mix(x):
    """A mixing of 32-bit numbers (in int64)."""
    m = 0xFFFFFFFF
    x = x ^ (x >> 16)
    x = (x * 0x7FEB352D) & m
    x = x ^ (x >> 15)
    x = (x * 0x846CA68B) & m
    return x ^ (x >> 16)


def _dither(n):
    """(int32, int32) 16 random bits each for the first and second moments of a tensor's n values."""
    key = _mix((_mix(0) + STEP) & 0xFFFFFFFF)
    bits = _mix(torch.arange(n, device=DEV) ^ _mix(key))
    return (bits >> 16).to(torch.int32), (bits & 0xFFFF).to(torch.int32)


def _code(value, dither):
    """(e4m3 bytes, scales) of values in groups of GROUP: value / scale, rounded to one of its neighbours by dither."""
    n = value.numel()
    rows = torch.nn.functional.pad(value, (0, -n % GROUP)).view(-1, GROUP)
    most = rows.abs().amax(-1, keepdim=True)
    y = (rows * torch.where(most > 0, 448 / most, 0)).view(-1)[:n]
    a = y.abs().clamp(max=448)
    base = torch.where(a < 2.0 ** -6, 2.0 ** -6, 0)
    kept = ((a + base).view(torch.int32) + (dither << 4)) & ~0xFFFFF
    c = torch.where(value != 0, (kept.view(torch.float32) - base).clamp(min=0), 0)
    return torch.copysign(c, y), (most / 448)[:, 0]


def _plain_update(s, i):
    """One tensor's update, in place."""
    c, p = s["case"], s["param"][i]
    master = s.get("master", {}).get(i)
    f = (p if master is None else master).float().view(-1)
    g, n = s["grad"][i].float().view(-1), p.numel()
    if c["bits"] == 8:
        of = torch.arange(n, device=DEV) // GROUP
        m = s["m"][i].float().view(-1) * s["m_scale"][i][of]
        v = (s["v"][i].float().view(-1) * s["v_scale"][i][of]).square()
    else:
        m, v = s["m"][i].view(-1), s["v"][i].view(-1)
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + g * g * (1 - BETA2)
    f = f * (1 - LR * DECAY) - LR / (1 - BETA1 ** STEP) * m / ((v / (1 - BETA2 ** STEP)).sqrt() + ADAM_EPS)
    p.view(-1).copy_(f)
    if master is not None:
        master.view(-1).copy_(f)
    if c["bits"] == 8:
        dm, dv = _dither(n)
        root = v.sqrt()
        m, scale = _code(m, dm)
        s["m_scale"][i].copy_(scale)
        v, scale = _code(root, dv)
        v = torch.where(root > 0, v.clamp(min=2.0 ** -9), 0)
        s["v_scale"][i].copy_(scale)
    s["m"][i].view(-1).copy_(m)
    s["v"][i].view(-1).copy_(v)


def _name(key):
    return key[0] + " " + str(key[1]).replace("torch.", "")


def _updated(flat):
    """The buffers that an update writes; 8-bit states as e4m3 values in units of their scales."""
    return {_name(k): t for k, t in flat.items() if k[0] != "grad"}


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "adamw":
        [_plain_update(s, i) for i in s["param"]]
        return _updated(s["flat"])
    if op == "gated":
        x = s["x"].float()
        g = (x @ s["w_gate"].float().T) * s["scale"]
        u = (x @ s["w_up"].float().T) * s["up_scale"]
        if c["bias"]:
            g, u = g + s["bias_gate"].float(), u + s["bias_up"].float()
        y = _act(c["act"], g) * u
        if c["out"] == "e4m3":
            r = {"y": (y * s["out_scale"]).clamp(-448, 448).to(torch.float8_e4m3fn)}
        else:
            r = {"y": y.to(TYPES[c["out"]])}
        if c["pre"]:
            kept = torch.bfloat16 if c["type"] == "e4m3" else s["x"].dtype
            r.update(pre_gate=g.to(kept), pre_up=u.to(kept))
        return r
    if op == "gated_grad":
        x, dy, g, u = s["x"].float(), s["dy"].float(), s["pre_gate"].float(), s["pre_up"].float()
        tg, tu = dy * u * _act_slope(c["act"], g), dy * _act(c["act"], g)
        dt = s["x"].dtype
        return {"dx": ((tg @ s["w_gate"].float()) * s["scale"] + (tu @ s["w_up"].float()) * s["up_scale"]).to(dt),
                "dw_gate": ((tg.T @ x) * s["scale"]).to(dt), "dw_up": ((tu.T @ x) * s["up_scale"]).to(dt),
                "dbias_gate": tg.sum(0), "dbias_up": tu.sum(0)}
    x, w, tok = s["x"].float(), s["w"].float(), s["tokens"]
    has = tok >= 0
    z = (x @ w.T) * s["scale"]
    if op == "head":
        m = z.amax(-1, keepdim=True)
        d = z - m
        e = torch.exp(d)
        total = e.sum(-1)
        lse = m[:, 0] + torch.log(total)
        lp = torch.where(has, z.gather(1, tok.clamp(min=0)[:, None])[:, 0] - lse, 0)
        return {"logprob": lp, "entropy": torch.log(total) - (e * d).sum(-1) / total, "lse": lse}
    logp = z - s["lse"][:, None]
    p = torch.exp(logp)
    dlp = torch.where(has, s["dlogprob"], 0)
    t = -p * dlp[:, None] - s["dentropy"][:, None] * p * (logp + s["entropy"][:, None])
    t.scatter_add_(1, tok.clamp(min=0)[:, None], dlp[:, None])
    return {"dx": ((t @ w) * s["scale"]).to(s["x"].dtype), "dw": ((t.T @ x) * s["scale"]).to(s["x"].dtype)}


# ------------------------------------------------------------------ the library's operators

def _kernels(s):
    import lossless_entropy_coding_gb300 as ecc

    c = s["case"]
    op = c["op"]
    if op == "adamw":
        lists = {k: list(s[k].values()) for k in ("param", "grad", "m", "v", "m_scale", "v_scale") if k in s}
        master = [s["master"].get(i) for i in s["param"]] if "master" in s else None
        state = ecc.AdamWState(lists["m"], lists["v"], lists.get("m_scale"), lists.get("v_scale"), master)
        ecc.ecc_adamw(lists["param"], lists["grad"], state, step=STEP, lr=LR, beta1=BETA1, beta2=BETA2, eps=ADAM_EPS,
                      weight_decay=DECAY, seed=0)
        return _updated(s["flat"])
    if op == "gated":
        kept = (None, None)
        if c["pre"]:
            kt = torch.bfloat16 if c["type"] == "e4m3" else s["x"].dtype
            kept = [torch.empty((c["M"], c["N"]), device=DEV, dtype=kt) for _ in range(2)]
        y, _ = ecc.ecc_gated_linear(s["x"], s["w_gate"], s["w_up"], s["bias_gate"], s["bias_up"], act=c["act"],
                                    scale=s["scale"], up_scale=s["up_scale"], out_dtype=TYPES[c["out"]],
                                    out_scale=s["out_scale"] if c["out"] == "e4m3" else 1.0,
                                    pre_gate=kept[0], pre_up=kept[1])
        return {"y": y, "pre_gate": kept[0], "pre_up": kept[1]} if c["pre"] else {"y": y}
    if op == "gated_grad":
        r = ecc.ecc_gated_linear_grad(s["dy"], s["x"], s["w_gate"], s["w_up"], s["pre_gate"], s["pre_up"],
                                      act=c["act"], scale=s["scale"], up_scale=s["up_scale"])
        return dict(zip(("dx", "dw_gate", "dw_up", "dbias_gate", "dbias_up"), r))
    if op == "head":
        r = ecc.ecc_linear_logprob(s["x"], s["w"], s["tokens"], scale=s["scale"])
        return {"logprob": r.logprob, "entropy": r.entropy, "lse": r.lse}
    dx, dw, _ = ecc.ecc_linear_logprob_grad(s["x"], s["w"], s["tokens"], s["lse"], s["entropy"], s["dlogprob"],
                                            s["dentropy"], scale=s["scale"])
    return {"dx": dx, "dw": dw}


def run(state):
    return _kernels(state) if own else _plain(state)


# ------------------------------------------------------------------ floors and exact values

def work(case):
    op = case["op"]
    if op == "adamw":
        total = 0
        rows = _layout(case)
        for shape, pt, gt, lo, n, at, groups in rows:
            total += n * (2 * pt.itemsize + gt.itemsize) + (4 * n + 16 * groups if case["bits"] == 8 else 16 * n)
            if case["master"] and pt != torch.float32:
                total += n * (8 - pt.itemsize)  # the master is read and written, the parameter only written
        return {"bytes": total, "flops": 14 * sum(row[4] for row in rows)}
    t, M, K = BYTES[case["type"]], case["M"], case["K"]
    if op == "gated":
        N = case["N"]
        each = BYTES[case["out"]] + (4 if case["pre"] else 0)
        return {"bytes": (M * K + 2 * N * K) * t + M * N * each + (4 * N if case["bias"] else 0),
                "flops": 4 * M * N * K}
    if op == "gated_grad":
        N = case["N"]
        return {"bytes": 2 * (M * K + 2 * N * K) * t + 3 * M * N * t + 8 * N, "flops": 8 * M * N * K}
    V = case["V"]
    if op == "head":
        return {"bytes": (M * K + V * K) * t + 20 * M, "flops": 2 * M * V * K}
    return {"bytes": 2 * (M * K + V * K) * t + 24 * M, "flops": 6 * M * V * K}


def _e4m3_neighbours(a):
    """The e4m3 values below and above magnitudes a (at most 448) and the part of the way between, in 64 bits."""
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -6))).clamp(max=8)
    ulp = torch.exp2(e - 3)
    low = torch.floor(a / ulp)
    return low * ulp, ulp, a / ulp - low


def _exact_code(value, bits16):
    """(values, scales) as the 8-bit states hold them: rounded up where the dither reaches over the remainder."""
    n = value.numel()
    groups = value.new_zeros((n + GROUP - 1) // GROUP * GROUP)
    groups[:n] = value.abs()
    scale = groups.view(-1, GROUP).max(-1).values / 448
    each = scale.repeat_interleave(GROUP)[:n]
    a = torch.where(each > 0, value.abs() / each, 0).clamp(max=448)
    low, ulp, part = _e4m3_neighbours(a)
    up = part * 65536 + bits16 >= 65536
    return torch.sign(value) * (low + torch.where(up, ulp, 0)), scale


def _exact_adamw(case, s):
    out = {k: t.double() for k, t in s["flat"].items() if k[0] != "grad"}
    for i, (shape, pt, gt, lo, n, at, groups) in enumerate(_layout(case)):
        mine = {k[0]: t[at:at + groups] if k[0].endswith("scale") else t[lo:lo + n] for k, t in out.items()
                if k[0] != "param" and (k[0] != "master" or pt != torch.float32)}
        param = out["param", pt][lo:lo + n]
        f, g = mine.get("master", param), s["flat"]["grad", gt][lo:lo + n].double()
        if case["bits"] == 8:
            each = [mine[k].repeat_interleave(GROUP)[:n] for k in ("m_scale", "v_scale")]
            m, v = mine["m"] * each[0], (mine["v"] * each[1]) ** 2
        else:
            m, v = mine["m"], mine["v"]
        m = torch.lerp(g, m, BETA1)
        v = torch.lerp(g ** 2, v, BETA2)
        step = (m / (1 - BETA1 ** STEP)) / (torch.sqrt(v / (1 - BETA2 ** STEP)) + ADAM_EPS)
        f.sub_(LR * (step + DECAY * f))
        param.copy_(f)
        if case["bits"] == 8:
            key = torch.tensor(0, device=DEV)
            for k in (0, STEP):  # the seed, then the step
                key = _mix((key + k) & 0xFFFFFFFF)
            bits = _mix(torch.arange(n, device=DEV) ^ _mix(key))
            positive = v > 0
            m, scale = _exact_code(m, bits // 65536)
            mine["m_scale"].copy_(scale)
            v, scale = _exact_code(v.sqrt(), bits % 65536)
            v = torch.where(positive, v.clamp(min=2.0 ** -9), 0)
            mine["v_scale"].copy_(scale)
        mine["m"].copy_(m)
        mine["v"].copy_(v)
    return {_name(k): t for k, t in out.items()}


def exact(case, seed):
    op = case["op"]
    # 64-bit products run at about 1e12 operations a second
    if op != "adamw" and work(case)["flops"] > 1.2e13:
        return None
    s = prepare(case, seed)
    if op == "adamw":
        return _exact_adamw(case, s)
    F = torch.nn.functional
    acts = {"none": lambda a: a, "relu": F.relu, "gelu": F.gelu, "silu": F.silu,
            "gelu_tanh": lambda a: F.gelu(a, approximate="tanh")}
    x = s["x"].double()
    if op == "gated":
        g, u = F.linear(x, s["w_gate"].double()) * s["scale"], F.linear(x, s["w_up"].double()) * s["up_scale"]
        if case["bias"]:
            g, u = g + s["bias_gate"].double(), u + s["bias_up"].double()
        y = acts[case["act"]](g) * u
        r = {"y": (y * s["out_scale"]).clamp(-448, 448) if case["out"] == "e4m3" else y}
        if case["pre"]:
            r.update(pre_gate=g, pre_up=u)
        return r
    if op == "gated_grad":
        g, u = s["pre_gate"].double().requires_grad_(), s["pre_up"].double().requires_grad_()
        tg, tu = torch.autograd.grad(acts[case["act"]](g) * u, (g, u), s["dy"].double())
        dx = torch.mm(tg, s["w_gate"].double()) * s["scale"]
        dx += torch.mm(tu, s["w_up"].double()) * s["up_scale"]
        return {"dx": dx, "dw_gate": torch.mm(tg.T, x) * s["scale"], "dw_up": torch.mm(tu.T, x) * s["up_scale"],
                "dbias_gate": tg.sum(0), "dbias_up": tu.sum(0)}
    w, got, dw = s["w"].double(), [], None
    step = max(1, (1 << 27) // w.shape[0])
    for i in range(0, x.shape[0], step):
        tok = s["tokens"][i:i + step]
        logp = torch.log_softmax(F.linear(x[i:i + step], w) * s["scale"], -1)
        ent = torch.special.entr(logp.exp()).sum(-1)
        has = torch.nonzero(tok >= 0)[:, 0]
        if op == "head":
            z = F.linear(x[i:i + step], w[:1])[:, 0] * s["scale"]
            lp = torch.zeros_like(ent)
            lp[has] = logp[has, tok[has]]
            got.append({"logprob": lp, "entropy": ent, "lse": z - logp[:, 0]})
            continue
        p = logp.exp()
        t = s["dentropy"][i:i + step].double()[:, None] * (-p * (logp + ent[:, None]))
        dlp = s["dlogprob"][i:i + step].double() * (tok >= 0)
        t -= p * dlp[:, None]
        t[has, tok[has]] += dlp[has]
        got.append({"dx": torch.mm(t, w) * s["scale"]})
        one = torch.mm(t.T, x[i:i + step]) * s["scale"]
        dw = one if dw is None else dw.add_(one)
    r = {k: torch.cat([o[k] for o in got]) for k in got[0]}
    if op == "head_grad":
        r["dw"] = dw
    return r
