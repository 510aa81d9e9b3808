"""AdamW: nothing that a call writes may overlap anything else that it is given,
what it only reads included (another warp would read it before or after it is
updated).  Refused before any CUDA call."""
import lossless_entropy_coding_gb300 as ecc
from test_lm_more_arguments import P, adamw, tensor

# tensor(at): parameter, m and v at 64 P at, + 8 P, + 16 P, of 1000 values (bf16, float32 states); gradients at P
N = 1000


def test_gradients_that_are_written():
    here = 64 * P
    for grad in (here, here + 2 * N - 2, here - 2 * N + 2, here + 8 * P, here + 8 * P + 4 * N - 4, here + 16 * P):
        assert adamw(tensor(grad=grad)) == ecc.ERR_ARG, grad
    # a gradient of one tensor in what another one updates, whichever comes first
    for a, b in ((tensor(1, grad=2 * here), tensor(2)), (tensor(1), tensor(2, grad=here + 8 * P + 2000)),
                 (tensor(1, master=500 * P), tensor(2, grad=500 * P + 3998)),
                 (tensor(1, grad_type=ecc.F32, grad=2 * here - 4 * N + 4), tensor(2))):
        assert adamw(a, b) == adamw(b, a) == ecc.ERR_ARG
    bytes_ = dict(state_type=ecc.E4M3, m_scale=400 * P, v_scale=401 * P)
    for grad in (400 * P, 400 * P + 14, 401 * P, here + 8 * P + N - 2):
        assert adamw(tensor(**bytes_, grad=grad)) == ecc.ERR_ARG, grad


def test_numbers_on_the_device_that_are_written():
    here = 64 * P
    for name, size in (("step_at", 8), ("lr_at", 4), ("grad_scale_at", 4)):
        for at in (here, here + 2 * N - size, here + 8 * P + 8, here + 16 * P + 4 * N - size):
            assert adamw(tensor(), **{name: at}) == ecc.ERR_ARG, (name, at)


def test_a_long_span_over_several_short_ones():
    # the overlap is not between neighbours in the order of addresses
    inside = [tensor(i, n=8, param=(300 + i) * P, m=(310 + i) * P, v=(320 + i) * P, grad=64 * P + i * 4096) for i in range(2, 5)]
    assert adamw(tensor(1, n=1 << 20), *inside) == ecc.ERR_ARG
    assert adamw(*inside, tensor(1, n=1 << 20)) == ecc.ERR_ARG
