"""The gated block of the coded feed-forward example: its operators together,
as a training step and a serving pass use them, against plain 64-bit torch."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import lossless_entropy_coding_gb300 as ecc  # noqa: E402
from examples import coded_ffn  # noqa: E402

F = torch.nn.functional


def plain(par, x):
    h = F.layer_norm(x, (x.shape[1],), par["n1"], par["c1"])
    a = F.gelu(F.linear(h, par["gate"]), approximate="tanh") * F.linear(h, par["up"])
    return F.linear(F.layer_norm(x + F.linear(a, par["down"]), (x.shape[1],), par["n2"], par["c2"]), par["head"])


def inputs(rows, width, vocab, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(rows, width, generator=g, device="cuda").to(torch.bfloat16)
    return x, torch.randint(0, vocab, (rows,), generator=g, device="cuda")


def test_it_runs_and_its_tensors_arrive_as_they_were_sent():
    served, history, moments = coded_ffn.run_gated(192, 256, 640, 1001, steps=3)
    assert served["lossless"] and moments["lossless"] and len(history) == 3
    assert served["activation_bits"] < 8 and moments["bits"] < 8 and all(math.isfinite(b) for b in history)


def test_the_step_follows_autograd_and_the_update_formula():
    rows, width, hidden, vocab = 96, 128, 320, 513
    par = coded_ffn.gated_parameters(width, hidden, vocab, seed=3)
    x, tokens = inputs(rows, width, vocab, 4)
    before = {k: v.clone() for k, v in par.items()}
    p = {k: v.double().requires_grad_() for k, v in before.items()}
    loss = F.cross_entropy(plain(p, x.double()), tokens)
    loss.backward()
    state = ecc.adamw_state(list(par.values()), 32)
    bits = coded_ffn.train_gated(x, tokens, par, state, 1, rate=1e-3)
    # five BF16 tensors between x and the logits, 2^-8 each, on logits of unit size
    assert abs(bits * math.log(2) - float(loss.detach())) < 5 * 2.0**-8 * 4
    for i, (k, v) in enumerate(par.items()):
        # the first moment is a tenth of the gradient, the second a twentieth of its square
        want = p[k].grad
        got = state.m[i].double() * 10
        assert float((got - want).norm()) < 0.03 * float(want.norm()) + 1e-6, k
        assert float((state.v[i].double() * 20 - got.square()).norm()) <= 1e-5 * float(got.square().norm()) + 1e-30
        # and the update its sign's: 1e-3, with the decay and half a step of BF16
        moved = before[k].double() * (1 - 1e-5) - par[k].double()
        step = 1e-3 * got / (got.abs() + 1e-8)
        half = 2.0**-8 if v.dtype == torch.bfloat16 else 2.0**-23
        assert bool(((moved - step).abs() <= half * (before[k].double().abs() + 1e-3) + 1e-7).all()), k


def test_eight_bit_moments_give_nearly_the_same_step():
    rows, width, hidden, vocab = 96, 128, 320, 513
    x, tokens = inputs(rows, width, vocab, 4)
    par = [coded_ffn.gated_parameters(width, hidden, vocab, seed=3) for _ in range(2)]
    state = [ecc.adamw_state(list(p.values()), bits) for p, bits in zip(par, (8, 32))]
    for p, s in zip(par, state):
        coded_ffn.train_gated(x, tokens, p, s, 1, rate=1e-3)
    for a, b in zip(par[0].values(), par[1].values()):
        assert torch.equal(a, b)                     # the first step's moments are used before they are rounded
    for i, m in enumerate(state[1].m):
        n = m.numel()
        scale = state[0].m_scale[i].repeat_interleave(ecc.ADAMW_GROUP)[:n]
        got = state[0].m[i].view(-1).view(torch.float8_e4m3fn).float() * scale
        # one of the two neighbours: at most a step of 2^-3 of the value, or 2^-9 of the scale
        assert bool(((got - m.view(-1)).abs() <= 2.0**-3 * m.view(-1).abs() * 1.001 + 2.0**-9 * scale * 1.001).all())


def test_serving_matches_the_plain_block_of_the_received_weights():
    rows, width, hidden, vocab = 130, 256, 512, 777
    par = coded_ffn.gated_parameters(width, hidden, vocab, seed=5)
    x, tokens = inputs(rows, width, vocab, 6)
    served = coded_ffn.serve_gated(x, tokens, par)
    q = {}
    for k, v in par.items():
        if v.dim() == 2:
            b, s = coded_ffn.e4m3(v.float())
            q[k] = b.view(torch.float8_e4m3fn).double() * s
        else:
            q[k] = v.double()
    loss = F.cross_entropy(plain(q, x.double()), tokens)
    # e4m3 rounding of three activations, 2^-4 each of logits of unit size, averaged over the text
    assert served["lossless"] and abs(served["bits_per_token"] * math.log(2) - float(loss)) < 3 * 2.0**-4
