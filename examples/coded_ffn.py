"""A feed-forward block and head whose tensors are coded as they move.

Serving: the weights arrive as entropy-coded e4m3 containers, are decoded and
multiplied; the hidden activation is written as e4m3 bytes by the matrix
product's epilogue, coded with a fixed Quad Length Code, decoded, and
multiplied again; the text's tokens get their log probabilities -- the model's
own code lengths -- and their most probable alternatives.

Training: one block in BF16 (layer norm, up projection with GELU, down
projection onto the residual stream, layer norm, head), the loss gradient from
the logits back to every parameter, and each weight gradient sent through the
BF16 exponent escape code before the update.

    python examples/coded_ffn.py
"""
import math
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import lossless_entropy_coding_gb300 as ecc  # noqa: E402

BF16, BYTES = torch.bfloat16, torch.uint8


def ok(*status):
    for s in status:
        if int(s.item()) != ecc.OK:
            raise RuntimeError(f"device status {int(s.item())}")


def sent(data, codebook):
    """data (e4m3 bytes) through an encode and a decode; (bytes received, coded bits)."""
    enc = ecc.ecc_encode(data.view(-1), ecc.to_device(codebook))
    out, st = ecc.ecc_decode(enc, ecc.to_device(codebook))
    ok(enc.status, st)
    return out[:data.numel()].view(data.shape), int(enc.total_bits.item())


def e4m3(x):
    """(bytes, scale): x as e4m3 bytes in units of its scale."""
    scale = float(x.abs().max()) / 256
    return (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(BYTES), scale


def book_of(data):
    """Quad Length Code adapted to a tensor's byte counts."""
    count = ecc.e4m3_histogram(data.view(-1))
    count = count.cpu().numpy().view(np.uint64)
    widths, _ = ecc.qlc_search_widths(count)
    return ecc.qlc_build_tables(count, widths)


def serve(x, tokens, w_up, b_up, w_down, b_down, w_head, top=5):
    """One pass over hidden states x [rows, width]; the dict says what came out and what it cost to send."""
    coded = raw = 0
    received = []
    for w in (w_up, w_down):                      # weights arrive coded
        q, scale = e4m3(w.float())
        q2, bits = sent(q, book_of(q))
        assert torch.equal(q2, q)
        received.append((q2, scale))
        coded, raw = coded + bits, raw + 8 * q.numel()
    (u, su), (d, sd) = received
    h, _, _ = ecc.ecc_layer_norm(x, out_dtype=BYTES, out_scale=16.0)
    calib, st = ecc.ecc_linear(h[:64], u, b_up, act="gelu", scale=su / 16, out_dtype=BYTES, out_scale=16.0)
    book = book_of(calib)                         # fixed before the batch is seen
    a, st2 = ecc.ecc_linear(h, u, b_up, act="gelu", scale=su / 16, out_dtype=BYTES, out_scale=16.0)
    ok(st, st2)
    a2, bits = sent(a, book)                      # the activation moves coded
    assert torch.equal(a2, a)
    y, st = ecc.ecc_linear(a2, d, b_down, residual=x, scale=sd / 16, out_dtype=BF16)
    z, _, _ = ecc.ecc_layer_norm(y)
    logits, st2 = ecc.ecc_linear(z, w_head)
    ok(st, st2)
    p = ecc.ecc_token_logprob(logits, tokens, top=top)
    return {"y": y, "activation": a, "activation_bits": bits / a.numel(), "weight_bits": 8 * coded / raw,
            "bits_per_token": float(-p.logprob.mean()) / math.log(2), "entropy_bits": float(p.entropy.mean()) / math.log(2),
            "top_index": p.top_index, "top_logprob": p.top_logprob, "logits": logits, "logprob": p.logprob}


def train_step(x, tokens, par, rate):
    """One step of the block on hidden states x; updates par; (bits per token, gradient bits a value)."""
    rows = x.shape[0]
    h, m1, r1 = ecc.ecc_layer_norm(x, par["n1"], par["c1"])
    pre = torch.empty(rows, par["up"].shape[0], dtype=BF16, device=x.device)
    a, s1 = ecc.ecc_linear(h, par["up"], par["bu"], act="gelu", pre=pre)
    y, s2 = ecc.ecc_linear(a, par["down"], par["bd"], residual=x)
    z, m2, r2 = ecc.ecc_layer_norm(y, par["n2"], par["c2"])
    logits, s3 = ecc.ecc_linear(z, par["head"])
    p = ecc.ecc_token_logprob(logits, tokens)
    bits = float(-p.logprob.mean()) / math.log(2)

    dlogp = torch.full((rows,), -1.0 / rows, device=x.device)   # the loss is the mean of -log p
    dlogits = ecc.ecc_token_logprob_grad(logits, tokens, p.lse, None, dlogp, dlogits=logits)
    g = {}
    dz, g["head"], _, s4 = ecc.ecc_linear_grad(dlogits, z, par["head"], want=("dx", "dw"))
    dy, g["n2"], g["c2"] = ecc.ecc_layer_norm_grad(dz, y, par["n2"], m2, r2)
    da, g["down"], g["bd"], s5 = ecc.ecc_linear_grad(dy, a, par["down"])
    dh, g["up"], g["bu"], s6 = ecc.ecc_linear_grad(da, h, par["up"], pre, act="gelu")
    _, g["n1"], g["c1"] = ecc.ecc_layer_norm_grad(dh, x, par["n1"], m1, r1)   # (dx = this + dy)
    ok(s1, s2, s3, s4, s5, s6)
    coded = values = 0
    for k, v in g.items():
        if v.dtype == BF16:                       # weight gradients move coded
            top7 = ecc.bf16_escape_table_sigma(max(float(v.float().std()), 1e-30))
            enc = ecc.bf16_escape_encode(v, top7)
            back, st = ecc.bf16_escape_decode(enc, top7)
            ok(enc.status, st)
            assert torch.equal(back[:v.numel()].view(BF16).view(v.shape), v)
            coded, values = coded + int(enc.total_bits.item()), values + v.numel()
        par[k] = (par[k].float() - rate * v.float()).to(par[k].dtype)
    return bits, coded / values


def serve_gated(x, tokens, par):
    """One pass of the gated block over hidden states x, weights and activation coded as they move."""
    received = {}
    for k in ("gate", "up", "down", "head"):
        q, scale = e4m3(par[k].float())
        q2, _ = sent(q, book_of(q))
        received[k] = (q2, scale)
    h, _, _ = ecc.ecc_layer_norm(x, par["n1"], par["c1"], out_dtype=BYTES, out_scale=16.0)
    (g, sg), (u, su), (d, sd), (w, sw) = (received[k] for k in ("gate", "up", "down", "head"))
    a, s1 = ecc.ecc_gated_linear(h, g, u, act="gelu_tanh", scale=sg / 16, up_scale=su / 16, out_dtype=BYTES, out_scale=16.0)
    a2, bits = sent(a, book_of(a[:64]))
    y, s2 = ecc.ecc_linear(a2, d, residual=x, scale=sd / 16, out_dtype=BF16)
    z, _, _ = ecc.ecc_layer_norm(y, par["n2"], par["c2"], out_dtype=BYTES, out_scale=16.0)
    p = ecc.ecc_linear_logprob(z, w, tokens, scale=sw / 16)
    ok(s1, s2, p.status)
    return {"activation_bits": bits / a.numel(), "bits_per_token": float(-p.logprob.mean()) / math.log(2), "lossless": torch.equal(a, a2)}


def train_gated(x, tokens, par, state, step, rate):
    """One step of the gated block under AdamW; updates par and state; bits per token."""
    rows = x.shape[0]
    h, m1, r1 = ecc.ecc_layer_norm(x, par["n1"], par["c1"])
    pre_g, pre_u = (torch.empty(rows, par["up"].shape[0], dtype=BF16, device=x.device) for _ in range(2))
    a, s1 = ecc.ecc_gated_linear(h, par["gate"], par["up"], act="gelu_tanh", pre_gate=pre_g, pre_up=pre_u)
    y, s2 = ecc.ecc_linear(a, par["down"], residual=x)
    z, m2, r2 = ecc.ecc_layer_norm(y, par["n2"], par["c2"])
    p = ecc.ecc_linear_logprob(z, par["head"], tokens)
    dlogp = torch.full((rows,), -1.0 / rows, device=x.device)   # the loss is the mean of -log p
    g = {}
    dz, g["head"], s3 = ecc.ecc_linear_logprob_grad(z, par["head"], tokens, p.lse, None, dlogp)
    dy, g["n2"], g["c2"] = ecc.ecc_layer_norm_grad(dz, y, par["n2"], m2, r2)
    da, g["down"], _, s4 = ecc.ecc_linear_grad(dy, a, par["down"], want=("dx", "dw"))
    dh, g["gate"], g["up"], _, _, s5 = ecc.ecc_gated_linear_grad(da, h, par["gate"], par["up"], pre_g, pre_u, act="gelu_tanh",
                                                                want=("dx", "dw"))
    _, g["n1"], g["c1"] = ecc.ecc_layer_norm_grad(dh, x, par["n1"], m1, r1)   # (dx = this + dy)
    ok(s1, s2, p.status, s3, s4, s5)
    for k, v in g.items():
        if v.dtype == BF16:                       # weight gradients move coded
            top7 = ecc.bf16_escape_table_sigma(max(float(v.float().std()), 1e-30))
            enc = ecc.bf16_escape_encode(v, top7)
            back, st = ecc.bf16_escape_decode(enc, top7)
            ok(enc.status, st)
            g[k] = back[:v.numel()].view(BF16).view(v.shape)
    ecc.ecc_adamw(list(par.values()), [g[k] for k in par], state, step, lr=rate, weight_decay=0.01, seed=1)
    return float(-p.logprob.mean()) / math.log(2)


def gated_parameters(width, hidden, vocab, device="cuda", seed=0):
    par = parameters(width, hidden, vocab, device, seed)
    gate = parameters(width, hidden, vocab, device, seed + 1)["up"]
    return {k: v for k, v in list(par.items()) + [("gate", gate)] if k not in ("bu", "bd")}


def run_gated(rows=512, width=512, hidden=2048, vocab=8000, steps=6, rate=2e-3):
    par = gated_parameters(width, hidden, vocab)
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(rows, width, generator=g, device="cuda").to(BF16)
    tokens = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    state = ecc.adamw_state(list(par.values()), bits=8)
    history = [train_gated(x, tokens, par, state, step + 1, rate) for step in range(steps)]
    moments = torch.cat([t.view(-1) for t in state.m + state.v])
    back, bits = sent(moments, book_of(moments))   # the optimizer's bytes, as for a checkpoint
    return serve_gated(x, tokens, par), history, {"lossless": torch.equal(back, moments), "bits": bits / moments.numel()}


def parameters(width, hidden, vocab, device="cuda", seed=0):
    g = torch.Generator(device).manual_seed(seed)

    def normal(*shape, std):
        return (torch.randn(shape, generator=g, device=device) * std).to(BF16)

    return {"n1": torch.ones(width, device=device), "c1": torch.zeros(width, device=device),
            "n2": torch.ones(width, device=device), "c2": torch.zeros(width, device=device),
            "up": normal(hidden, width, std=width**-0.5), "bu": torch.zeros(hidden, device=device),
            "down": normal(width, hidden, std=hidden**-0.5), "bd": torch.zeros(width, device=device),
            "head": normal(vocab, width, std=width**-0.5)}


def run(rows=512, width=512, hidden=2048, vocab=8000, steps=6, rate=2.0):
    par = parameters(width, hidden, vocab)
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(rows, width, generator=g, device="cuda").to(BF16)
    tokens = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    served = serve(x, tokens, par["up"], par["bu"], par["down"], par["bd"], par["head"])
    history = [train_step(x, tokens, par, rate) for _ in range(steps)]
    return served, history


if __name__ == "__main__":
    served, history = run()
    print(f"serving: weights {served['weight_bits']:.2f} bits a value, activation {served['activation_bits']:.2f}, "
          f"text {served['bits_per_token']:.2f} bits a token (entropy {served['entropy_bits']:.2f})")
    for i, (bits, grad) in enumerate(history):
        print(f"step {i}: {bits:.3f} bits a token, weight gradients {grad:.2f} bits a value")
    served, history, moments = run_gated()
    for i, bits in enumerate(history):
        print(f"gated block, step {i}: {bits:.3f} bits a token")
    print(f"served: {served['bits_per_token']:.3f} bits a token, activation {served['activation_bits']:.2f} bits a value, "
          f"AdamW's moments {moments['bits']:.2f}")
