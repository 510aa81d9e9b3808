"""The Python side of AdamW, without a GPU: which device a stream has to belong to."""
from types import SimpleNamespace

import pytest

import lossless_entropy_coding_gb300 as ecc

torch = pytest.importorskip("torch")


def test_a_stream_of_another_device_than_the_tensors_that_are_updated():
    a, b, x = torch.device("cuda:0"), torch.device("cuda:1"), torch.zeros(4)
    here, there = SimpleNamespace(device=a), SimpleNamespace(device=b)
    state = ecc.AdamWState([x, x], [x, x])
    for params, grads in (([here, there], [None, x]), ([there, here], [x, None]), ([there, there], [x, x]), ((here, there), (None, x))):
        with pytest.raises(ecc.EccError, match="stream of another device"):
            ecc.ecc_adamw(params, grads, state, step=1, stream=SimpleNamespace(device=a))
    for params, grads in ((x, [x]), ([x], x), (None, None), ([x], [x])):     # lists, and tensors of a GPU
        with pytest.raises(ecc.EccError):
            ecc.ecc_adamw(params, grads, state, step=1, stream=SimpleNamespace(device=a))


def test_masters_are_apart_from_autograd():
    params = [torch.nn.Parameter(torch.randn(5).to(t)) for t in (torch.bfloat16, torch.float16, torch.float32)]
    params.append((params[0] * 2))                        # with a graph behind it
    state = ecc.adamw_state(params, 8, master=True)
    for p, m in zip(params, state.master):
        if p.dtype == torch.float32:
            assert m is None
        else:
            assert m.dtype == torch.float32 and not m.requires_grad and m.grad_fn is None and torch.equal(m, p.detach().float())


def test_a_state_for_any_iterable_of_parameters():
    layer = torch.nn.Linear(300, 5).to(torch.bfloat16)
    for bits, master in ((32, False), (32, True), (8, False), (8, True)):
        want, got = (ecc.adamw_state(p, bits, master) for p in (list(layer.parameters()), layer.parameters()))
        for a, b in zip(want, got):
            assert (a is None) == (b is None)
            assert a is None or (len(a) == len(b) == 2 and all(p.shape == q.shape and p.dtype == q.dtype for p, q in zip(a, b)))
