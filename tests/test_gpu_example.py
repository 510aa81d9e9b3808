"""The coded feed-forward example: its tensors arrive as they were sent, its
results are those of the same block in plain torch, and training lowers the
code length of the text."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from examples import coded_ffn  # noqa: E402


def test_serving_and_training_run_together():
    rows, width, hidden, vocab = 192, 256, 640, 1001
    served, history = coded_ffn.run(rows, width, hidden, vocab, steps=5, rate=1.0)
    # the code words of the fitted layouts are shorter than the bytes
    assert served["weight_bits"] < 8 and served["activation_bits"] < 8
    # the text's code length and entropy follow from the logits alone
    z = served["logits"].double()
    logp = torch.log_softmax(z, -1)
    ent = -(logp.exp() * logp).sum(-1).mean() / math.log(2)
    assert abs(float(ent) - served["entropy_bits"]) < 1e-4
    top = torch.sort(served["logits"].float(), dim=-1, descending=True, stable=True).indices[:, :5]
    assert torch.equal(served["top_index"].long(), top)
    # the training step's first loss is the plain block's (BF16 tensors between the operators: 2^-8 each)
    par = coded_ffn.parameters(width, hidden, vocab)
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(rows, width, generator=g, device="cuda").to(torch.bfloat16)
    tokens = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    F = torch.nn.functional
    p = {k: v.double() for k, v in par.items()}
    xd = x.double()
    h = F.layer_norm(xd, (width,), p["n1"], p["c1"])
    y = xd + F.linear(F.gelu(F.linear(h, p["up"], p["bu"])), p["down"], p["bd"])
    logits = F.linear(F.layer_norm(y, (width,), p["n2"], p["c2"]), p["head"])
    loss = F.cross_entropy(logits, tokens) / math.log(2)
    assert abs(float(loss) - history[0][0]) < 0.05
    assert history[-1][0] < history[0][0] - 0.5
    assert all(grad < 16 for _, grad in history)


def test_training_step_gradients_match_autograd():
    rows, width, hidden, vocab = 96, 128, 320, 513
    par = coded_ffn.parameters(width, hidden, vocab, seed=3)
    before = {k: v.clone() for k, v in par.items()}
    g = torch.Generator("cuda").manual_seed(4)
    x = torch.randn(rows, width, generator=g, device="cuda").to(torch.bfloat16)
    tokens = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    rate = 512.0                       # a power of two large enough that the update shows in BF16 weights
    coded_ffn.train_step(x, tokens, par, rate)
    F = torch.nn.functional
    p = {k: v.double().requires_grad_() for k, v in before.items()}
    xd = x.double()
    h = F.layer_norm(xd, (width,), p["n1"], p["c1"])
    y = xd + F.linear(F.gelu(F.linear(h, p["up"], p["bu"])), p["down"], p["bd"])
    logits = F.linear(F.layer_norm(y, (width,), p["n2"], p["c2"]), p["head"])
    F.cross_entropy(logits, tokens).backward()
    for k in par:
        got = (before[k].double() - par[k].double()) / rate
        want = p[k].grad
        # BF16 tensors between the operators and the update rounded to BF16
        assert float((got - want).norm()) < 0.03 * float(want.norm()) + 1e-6, k
