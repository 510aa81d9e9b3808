"""The Python entry points of the language-model operators take their
arguments by position and by name (checked without a GPU: a host tensor is
refused by the operator, after the arguments have found their places)."""
import pytest

torch = pytest.importorskip("torch")

import lossless_entropy_coding_gb300 as ecc  # noqa: E402

x = torch.zeros(2, 8)
CALLS = {
    "ecc_layer_norm": dict(x=x),
    "ecc_layer_norm_grad": dict(dy=x, x=x, weight=None, mean=x[:, 0], rstd=x[:, 0]),
    "ecc_linear": dict(x=x, w=x),
    "ecc_linear_grad": dict(dy=x, x=x, w=x),
    "ecc_token_logprob": dict(logits=x, tokens=None),
    "ecc_token_logprob_grad": dict(logits=x, tokens=None, lse=x[:, 0]),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_arguments_by_name_and_by_position(name):
    f, args = getattr(ecc, name), CALLS[name]
    for n in range(len(args) + 1):        # the first n by position
        with pytest.raises(ecc.EccError) as e:
            f(*list(args.values())[:n], **dict(list(args.items())[n:]))
        assert e.value.code == ecc.ERR_ARG
    with pytest.raises(TypeError):
        f()
    with pytest.raises(TypeError):
        f(**args, other=1)
