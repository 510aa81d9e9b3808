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
