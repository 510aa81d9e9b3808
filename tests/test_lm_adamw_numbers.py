"""AdamW's numbers are used in float32: what has no finite value there is
refused, before any CUDA call."""
import pytest

import lossless_entropy_coding_gb300 as ecc
from test_lm_more_arguments import adamw, tensor


@pytest.mark.parametrize("name", ["lr", "eps", "weight_decay", "grad_scale"])
@pytest.mark.parametrize("value", [1e39, 3.5e38, 1e300])
def test_numbers_beyond_float32(name, value):
    assert adamw(tensor(), **{name: value}) == ecc.ERR_ARG
    if name != "eps":
        assert adamw(tensor(), **{name: -value}) == ecc.ERR_ARG
