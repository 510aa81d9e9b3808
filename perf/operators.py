"""The language-model operators next to the coders, as timed workloads: layer
norm, the matrix product with a fused epilogue, and token log probabilities,
each with its gradient.

`run` computes a case either in plain torch operations (own = False) or with
the library's kernels (own = True); `exact` gives the same outputs in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}
EPS = 1e-5
# a drawn case costs at most what the largest listed one of its operator does
NORM_MOST, LINEAR_MOST, LOGPROB_MOST = 16384 * 4096, 8192 * 4096 * 16384, 4096 * 131072


def listed():
    return [
        # a decode step's normalisation of a few sequences: latency
        dict(name="norm step", op="norm", rows=4, cols=2048, pad=0, type="bf16", out="bf16"),
        # a prompt's normalisation into the e4m3 operand of the next product
        dict(name="norm prompt e4m3", op="norm", rows=16384, cols=4096, pad=0, type="bf16", out="e4m3"),
        # a training batch's backward pass, with the reduction over its tokens
        dict(name="norm grad", op="norm_grad", rows=16384, cols=4096, pad=0, type="bf16"),
        # one token through the up projection: the weights are read once
        dict(name="linear token", op="linear", M=1, N=16384, K=4096, pad=0, type="bf16", out="bf16", act="gelu",
             bias=True, residual=False, pre=False),
        # a training batch through the up projection, pre-activation kept for the backward pass
        dict(name="linear up", op="linear", M=8192, N=16384, K=4096, pad=0, type="bf16", out="bf16", act="gelu",
             bias=True, residual=False, pre=True),
        # the down projection of decoded e4m3 activations and weights, added to the residual stream
        dict(name="linear down e4m3", op="linear", M=2048, N=4096, K=16384, pad=0, type="e4m3", out="bf16",
             act="none", bias=True, residual=True, pre=False),
        # odd sizes, rows that start anywhere
        dict(name="linear ragged", op="linear", M=333, N=1111, K=1001, pad=0, type="f16", out="f16", act="silu",
             bias=True, residual=True, pre=True),
        # the up projection's backward pass for a training batch
        dict(name="linear grad", op="linear_grad", M=8192, N=16384, K=4096, pad=0, type="bf16", act="gelu"),
        # a small layer's backward pass on a ragged batch
        dict(name="linear grad ragged", op="linear_grad", M=257, N=1000, K=770, pad=0, type="f16",
             act="gelu_tanh"),
        # a decode step of a few sequences: the sampled tokens' log probabilities and their alternatives
        dict(name="logprob step", op="logprob", rows=8, vocab=131072, pad=0, type="bf16", scale=1.0, top=8),
        # scoring a text under a vocabulary of odd size
        dict(name="logprob score", op="logprob", rows=4096, vocab=50021, pad=0, type="f32", scale=0.7, top=20),
        # the loss gradient of a training batch
        dict(name="logprob grad", op="logprob_grad", rows=4096, vocab=131072, pad=0, type="bf16", scale=1.0),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]: odd, a multiple of 8 or of 64."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    kind = rng.randrange(3)
    v = v | 1 if kind == 0 else v // 8 * 8 if kind == 1 else v // 64 * 64
    return min(hi, max(lo, v))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "linear", "linear", "linear_grad", "logprob", "logprob_grad"])
    pad = rng.choice([0, 0, 8, 5])
    if op in ("norm", "norm_grad"):
        cols = _log(rng, 48, 16384)
        c = dict(op=op, rows=_log(rng, 1, min(65536, NORM_MOST // cols)), cols=cols, pad=pad,
                 type=rng.choice(["bf16", "f16", "f32"]))
        if op == "norm":
            c["out"] = rng.choice([c["type"], "e4m3"])
        return c
    if op in ("linear", "linear_grad"):
        most = LINEAR_MOST if op == "linear_grad" else LINEAR_MOST // 2
        N, K = _log(rng, 64, 16384), _log(rng, 64, 16384)
        c = dict(op=op, M=_log(rng, 1, max(1, min(8192, most // (N * K)))), N=N, K=K, pad=pad,
                 type=rng.choice(["bf16", "f16"] if op == "linear_grad" else ["bf16", "f16", "e4m3"]),
                 act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]))
        if op == "linear":
            c.update(bias=rng.random() < 0.7, residual=rng.random() < 0.4, pre=rng.random() < 0.3)
            c["out"] = rng.choice(["bf16", "e4m3"] if c["type"] == "e4m3" else [c["type"], c["type"], "f32"])
        return c
    V = _log(rng, 1000, 262144)
    c = dict(op=op, rows=_log(rng, 1, min(8192, LOGPROB_MOST // V)), vocab=V, pad=pad,
             type=rng.choice(["bf16", "f16", "f32"]), scale=rng.choice([1.0, 0.7, 1.4]))
    if op == "logprob":
        c["top"] = rng.choice([0, 1, 5, 20, 32])
    return c


# ------------------------------------------------------------------ inputs

def _normal(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(dtype)


def _rows(g, rows, cols, pad, dtype, std=1.0):
    """[rows, cols] values in rows of cols + pad elements."""
    if dtype == torch.float8_e4m3fn:
        t = _normal(g, rows, cols + pad, std=std).clamp(-448, 448).to(dtype)
    else:
        t = _normal(g, rows, cols + pad, std=std, dtype=dtype)
    return t[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, pad, dt = case["op"], case["pad"], TYPES[case["type"]]
    s = dict(case=case)
    if op in ("norm", "norm_grad"):
        rows, cols = case["rows"], case["cols"]
        x = _rows(g, rows, cols, pad, dt)
        # a few channels far larger than the rest, as a residual stream has
        far = torch.randint(0, cols, (max(1, cols // 256),), generator=g, device=DEV)
        x[:, far] *= 20
        s.update(x=x, weight=(1 + _normal(g, cols, std=0.2)).to(dt), bias=_normal(g, cols, std=0.2, dtype=dt))
        if op == "norm_grad":
            xf = x.float()
            mean = xf.mean(-1)
            s.update(dy=_rows(g, rows, cols, pad, dt), mean=mean,
                     rstd=torch.rsqrt((xf - mean[:, None]).square().mean(-1) + EPS))
    elif op in ("linear", "linear_grad"):
        M, N, K = case["M"], case["N"], case["K"]
        x = _rows(g, M, K, pad, dt)
        if dt == torch.float8_e4m3fn:  # weights in units of their scale
            w, s["scale"] = _rows(g, N, K, pad, dt, std=16.0), 1 / (16.0 * math.sqrt(K))
        else:
            w, s["scale"] = _rows(g, N, K, pad, dt, std=1 / math.sqrt(K)), 1.0
        s.update(x=x, w=w)
        if op == "linear":
            od = torch.bfloat16 if case["out"] == "e4m3" else TYPES[case["out"]]
            s.update(bias=_normal(g, N, std=0.5, dtype=torch.bfloat16 if dt.itemsize == 1 else dt)
                     if case["bias"] else None,
                     residual=_rows(g, M, N, pad, od) if case["residual"] else None, out_scale=4.0)
        else:
            s.update(dy=_rows(g, M, N, pad, dt, std=0.1),
                     pre=_rows(g, M, N, pad, dt) if case["act"] != "none" else None)
    else:
        rows, V = case["rows"], case["vocab"]
        z = _rows(g, rows, V, pad, dt, std=2.5)
        z[:, V - V // 200:] = -math.inf  # the end of the vocabulary is padding
        tok = torch.randint(0, V - V // 200, (rows,), generator=g, device=DEV)
        tok[torch.rand(rows, generator=g, device=DEV) < 0.05] = -1  # positions without a token
        s.update(logits=z, tokens=tok)
        if op == "logprob_grad":
            lse = torch.logsumexp(z.float() * case["scale"], -1)
            p = torch.softmax(z.float() * case["scale"], -1)
            ent = lse - (p * torch.where(p > 0, z.float() * case["scale"], 0)).sum(-1)
            s.update(lse=lse, entropy=ent, dlogprob=-(torch.rand(rows, generator=g, device=DEV) + 0.5),
                     dentropy=_normal(g, rows, std=0.1))
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


def _store(y, out, scale):
    if out == "e4m3":
        return (y * scale).clamp(-448, 448).to(torch.float8_e4m3fn)
    return y.to(TYPES[out])


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "norm":
        x = s["x"].float()
        mean = x.mean(-1, keepdim=True)
        rstd = torch.rsqrt((x - mean).square().mean(-1, keepdim=True) + EPS)
        y = (x - mean) * rstd * s["weight"].float() + s["bias"].float()
        return {"y": _store(y, c["out"], 16.0), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    if op == "norm_grad":
        x, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
        xh = (x - s["mean"][:, None]) * rstd
        gw = dy * s["weight"].float()
        dx = rstd * (gw - gw.mean(-1, keepdim=True) - xh * (gw * xh).mean(-1, keepdim=True))
        return {"dx": dx.to(s["x"].dtype), "dweight": (dy * xh).sum(0), "dbias": dy.sum(0)}
    if op == "linear":
        a = (s["x"].float() @ s["w"].float().T) * s["scale"]
        if s["bias"] is not None:
            a = a + s["bias"].float()
        y = _act(c["act"], a)
        if s["residual"] is not None:
            y = y + s["residual"].float()
        r = {"y": _store(y, c["out"], s["out_scale"])}
        if c["pre"]:
            r["pre"] = a.to(torch.bfloat16 if c["type"] == "e4m3" else s["x"].dtype)
        return r
    if op == "linear_grad":
        t = s["dy"].float()
        if s["pre"] is not None:
            t = t * _act_slope(c["act"], s["pre"].float())
        return {"dx": ((t @ s["w"].float()) * s["scale"]).to(s["x"].dtype),
                "dw": ((t.T @ s["x"].float()) * s["scale"]).to(s["x"].dtype), "dbias": t.sum(0)}
    z = s["logits"].float() * c["scale"]
    tok = s["tokens"]
    has = tok >= 0
    if op == "logprob":
        m = z.amax(-1, keepdim=True)
        d = z - m
        e = torch.exp(d)
        total = e.sum(-1)
        lse = m[:, 0] + torch.log(total)
        ent = torch.log(total) - torch.where(e > 0, e * d, 0).sum(-1) / total
        lp = torch.where(has, z.gather(1, tok.clamp(min=0)[:, None])[:, 0] - lse, 0)
        r = {"logprob": lp, "entropy": ent, "lse": lse}
        if c["top"]:
            # one whole-number key of a value and its place: larger values first, then lower places
            b = torch.where(z == 0, 0.0, z).view(torch.int32).to(torch.int64)
            b = torch.where(b < 0, -(b & 0x7FFFFFFF), b)
            at = torch.arange(z.shape[1], device=z.device)
            key = (b << 20) + (0xFFFFF - at)
            idx = 0xFFFFF - (key.topk(c["top"], -1).values & 0xFFFFF)
            r["top_logprob"] = z.gather(1, idx) - lse[:, None]
            r["top_index"] = idx.to(torch.int32)
        return r
    logp = z - s["lse"][:, None]
    p = torch.exp(logp)
    dlp = torch.where(has, s["dlogprob"], 0)
    d = -p * dlp[:, None] - s["dentropy"][:, None] * torch.where(p > 0, p * (logp + s["entropy"][:, None]), 0)
    d.scatter_add_(1, tok.clamp(min=0)[:, None], dlp[:, None])
    return {"dlogits": (d * c["scale"]).to(s["logits"].dtype)}


# ------------------------------------------------------------------ the library's operators

def _kernels(s):
    import lossless_entropy_coding_gb300 as ecc

    c = s["case"]
    op = c["op"]
    if op == "norm":
        y, mean, rstd = ecc.ecc_layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, out_dtype=TYPES[c["out"]],
                                           out_scale=16.0 if c["out"] == "e4m3" else 1.0)
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_grad":
        dx, dw, db = ecc.ecc_layer_norm_grad(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"])
        return {"dx": dx, "dweight": dw, "dbias": db}
    if op == "linear":
        pre = None
        if c["pre"]:
            pre = torch.empty((c["M"], c["N"]), device=DEV,
                              dtype=torch.bfloat16 if c["type"] == "e4m3" else s["x"].dtype)
        y, _ = ecc.ecc_linear(s["x"], s["w"], s["bias"], s["residual"], act=c["act"], scale=s["scale"],
                              out_dtype=TYPES[c["out"]], out_scale=s["out_scale"] if c["out"] == "e4m3" else 1.0,
                              pre=pre)
        return {"y": y, "pre": pre} if c["pre"] else {"y": y}
    if op == "linear_grad":
        dx, dw, db, _ = ecc.ecc_linear_grad(s["dy"], s["x"], s["w"], s["pre"], act=c["act"], scale=s["scale"])
        return {"dx": dx, "dw": dw, "dbias": db}
    if op == "logprob":
        r = ecc.ecc_token_logprob(s["logits"], s["tokens"], top=c["top"], scale=c["scale"])
        d = {"logprob": r.logprob, "entropy": r.entropy, "lse": r.lse}
        if c["top"]:
            d.update(top_logprob=r.top_logprob, top_index=r.top_index)
        return d
    return {"dlogits": ecc.ecc_token_logprob_grad(s["logits"], s["tokens"], s["lse"], s["entropy"], s["dlogprob"],
                                                  s["dentropy"], scale=c["scale"])}


def run(state):
    return _kernels(state) if own else _plain(state)


# ------------------------------------------------------------------ floors and exact values

def work(case):
    op, t = case["op"], BYTES[case["type"]]
    if op in ("norm", "norm_grad"):
        n = case["rows"] * case["cols"]
        if op == "norm":
            return {"bytes": n * (t + BYTES[case["out"]]) + 2 * t * case["cols"] + 8 * case["rows"], "flops": 8 * n}
        return {"bytes": 3 * n * t + (t + 8) * case["cols"] + 8 * case["rows"], "flops": 14 * n}
    if op in ("linear", "linear_grad"):
        M, N, K = case["M"], case["N"], case["K"]
        if op == "linear":
            out = 2 if case["out"] == "e4m3" else BYTES[case["out"]]
            each = BYTES[case["out"]] + (out if case["residual"] else 0) + (2 if case["pre"] else 0)
            return {"bytes": (M * K + N * K) * t + M * N * each + (2 * N if case["bias"] else 0),
                    "flops": 2 * M * N * K}
        return {"bytes": 2 * (M * K + N * K) * t + M * N * t * (1 if case["act"] == "none" else 2) + 4 * N,
                "flops": 4 * M * N * K}
    n = case["rows"] * case["vocab"]
    if op == "logprob":
        return {"bytes": n * t + case["rows"] * (20 + 8 * case["top"]), "flops": 6 * n}
    return {"bytes": 2 * n * t + case["rows"] * 24, "flops": 8 * n}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    F = torch.nn.functional
    acts = {"none": lambda a: a, "relu": F.relu, "gelu": F.gelu, "silu": F.silu,
            "gelu_tanh": lambda a: F.gelu(a, approximate="tanh")}

    def stored(y, scale):
        return (y * scale).clamp(-448, 448) if case["out"] == "e4m3" else y

    if op == "norm":
        x = s["x"].double()
        var, mean = torch.var_mean(x, -1, correction=0)
        y = F.layer_norm(x, x.shape[-1:], s["weight"].double(), s["bias"].double(), EPS)
        return {"y": stored(y, 16.0), "mean": mean, "rstd": (var + EPS).rsqrt()}
    if op == "norm_grad":
        x, w = s["x"].double().requires_grad_(), s["weight"].double().requires_grad_()
        b = torch.zeros_like(w, requires_grad=True)
        F.layer_norm(x, x.shape[-1:], w, b, EPS).backward(s["dy"].double())
        return {"dx": x.grad, "dweight": w.grad, "dbias": b.grad}
    if op == "linear":
        a = F.linear(s["x"].double(), s["w"].double()) * s["scale"]
        a = a if s["bias"] is None else a + s["bias"].double()
        y = acts[case["act"]](a)
        y = y if s["residual"] is None else y + s["residual"].double()
        return {"y": stored(y, s["out_scale"]), "pre": a} if case["pre"] else {"y": stored(y, s["out_scale"])}
    if op == "linear_grad":
        t = s["dy"].double()
        if s["pre"] is not None:
            a = s["pre"].double().requires_grad_()
            t, = torch.autograd.grad(acts[case["act"]](a), a, t)
        return {"dx": torch.mm(t, s["w"].double()) * s["scale"],
                "dw": torch.mm(t.T, s["x"].double()) * s["scale"], "dbias": t.sum(0)}
    rows, got = s["logits"].shape[0], []
    step = max(1, (1 << 26) // s["logits"].shape[1])
    for i in range(0, rows, step):
        z = s["logits"][i:i + step].double().mul(case["scale"]).requires_grad_()
        tok = s["tokens"][i:i + step]
        logp = torch.log_softmax(z, -1)
        ent = torch.special.entr(logp.exp()).sum(-1)
        lp = torch.where(tok >= 0, logp.gather(1, tok.clamp(min=0)[:, None])[:, 0], 0)
        if op == "logprob":
            with torch.no_grad():
                one = {"logprob": lp, "entropy": ent, "lse": torch.logsumexp(z, -1)}
                if case["top"]:
                    one["top_logprob"] = logp.topk(case["top"], -1).values
                got.append({k: v.detach() for k, v in one.items()})
            continue
        # d entropy / d z = -p (log p + H), written out: log p is infinite where the logit is masked
        with torch.no_grad():
            p = logp.exp()
            d = -p * torch.where(tok >= 0, s["dlogprob"][i:i + step], 0).double()[:, None]
            d -= s["dentropy"][i:i + step].double()[:, None] * torch.where(p > 0, p * (logp + ent[:, None]), 0)
            has = torch.nonzero(tok >= 0)[:, 0]
            d[has, tok[has]] += s["dlogprob"][i:i + step][has].double()
            got.append({"dlogits": d * case["scale"]})
    r = {k: torch.cat([x[k] for x in got]) for k in got[0]}
    if op == "logprob" and case["top"]:
        r["top_index"] = None
    return r
