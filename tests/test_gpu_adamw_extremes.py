"""AdamW where float32's range ends: gradients whose squares are infinite, groups
of 8-bit states whose largest value is next to nothing.

The second moment is then infinity in float32, its root too, and the step
m / (root + eps) zero: the parameter only decays.  Tolerance: p (1 - lr
weight_decay) is two roundings of 2^-24, and half a step of the parameter's
type.  A group's codes are within a step of e4m3 of value / scale, which is
off by 2^-21 of itself.  Scales below float32's smallest normal value (2^-126)
have a rounding of 2^-150 more, relative to at least 2^-119 / 448: 2^-22."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import lossless_entropy_coding_gb300 as ecc  # noqa: E402
import test_gpu_adamw as adamw  # noqa: E402

F32, BF16, BYTE, E4M3, G = torch.float32, torch.bfloat16, torch.uint8, torch.float8_e4m3fn, ecc.ADAMW_GROUP
HYPER = adamw.HYPER


@pytest.mark.parametrize("skew", [0, 3])
@pytest.mark.parametrize("ptype,gtype,bits,master", [(F32, F32, 32, False), (BF16, BF16, 32, True), (BF16, F32, 8, True), (F32, BF16, 8, False)])
@pytest.mark.parametrize("size,grad_scale", [(1e20, 1.0), (-3e38, 1.0), (2e10, 1e10)])
def test_squares_beyond_the_range(ptype, gtype, bits, master, size, grad_scale, skew):
    n = 4 * G + 100
    p, g, state = adamw.make(n, ptype, gtype, bits, master, skew=skew)
    far = torch.zeros(n, dtype=torch.bool, device="cuda")
    far[[5, G + 1, G + 2, n - 1]] = True
    groups = torch.tensor([True, True, False, False, True], device="cuda")
    g /= grad_scale
    clean = g.clone()
    g[far] = size
    values = state.master[0] if master else p
    for step in (1, 2, 3):
        old_p, old, was = p.clone(), adamw.copied(state), values.clone()
        q, s2 = p.clone(), adamw.copied(state)
        ecc.ecc_adamw([p], [g], state, step=step, grad_scale=grad_scale, **HYPER)
        ecc.ecc_adamw([q], [clean], s2, step=step, grad_scale=grad_scale, **HYPER)
        want = was.double()[far] * (1 - HYPER["lr"] * HYPER["weight_decay"])
        assert bool(((values.double()[far] - want).abs() <= (2.0**-22 + torch.finfo(values.dtype).eps / 2) * want.abs()).all())
        if bits == 32:
            assert bool(torch.isinf(state.v[0][far]).all()) and bool(torch.isfinite(state.m[0]).all())
            assert torch.equal(p[~far], q[~far]) and torch.equal(state.v[0][~far], s2.v[0][~far])
            # (the others' moments are the clean ones: the next steps start from them)
        else:
            assert torch.equal(torch.isnan(state.v_scale[0]), groups) and torch.equal(torch.isnan(state.m_scale[0]), groups)
            whole = ~groups.repeat_interleave(G)[:n]
            assert torch.equal(p[~far], q[~far]) and torch.equal(state.m[0][whole], s2.m[0][whole])
            break                                        # (a group of NaN stays one)


@pytest.mark.parametrize("skew", [0, 3])
@pytest.mark.parametrize("top", [0.9e-36, 1.05e-36, 1.1e-36, 1.3e-36, 1.32e-36, 2.0**-119, 1.6e-36, 3e-36, 1e-35, 1e-30])
def test_groups_of_next_to_nothing(top, skew):
    """m = (1 - beta1) g of at most `top`: codes and scale hold it from 2^-119 on, below that the codes are zeros."""
    n = 2 * G + 60
    p, g, state = (torch.zeros(n + 16, dtype=t, device="cuda")[skew:skew + n] for t in (F32, F32, BYTE))
    state = ecc.AdamWState([state], [state.clone()], [torch.zeros(3, device="cuda")], [torch.zeros(3, device="cuda")])
    gen = torch.Generator("cuda").manual_seed(1)
    share = torch.rand(n, generator=gen, device="cuda") * 2 - 1
    share[[0, G, 2 * G]] = 1.0
    share[[1, G + 7, 2 * G + 3]] = 0.0
    m = (share.double() * top).float()
    g.copy_(m)
    ecc.ecc_adamw([p], [g], state, step=1, beta1=0.0, lr=0.0, seed=3)
    value = state.m[0].view(E4M3).double()
    assert not bool(state.v[0].any()) and not bool(p.any())
    if float(m[0]) < 2.0**-119:
        assert not bool(value.any())
        return
    scale = m[0].double() / 448
    assert bool(((state.m_scale[0].double() - scale).abs() <= 2.0**-21 * scale).all())
    assert bool((value[[0, G, 2 * G]] == 448).all()) and not bool(value[[1, G + 7, 2 * G + 3]].any())
    want = (m.double() / scale).clamp(-448, 448)
    step = torch.exp2(torch.floor(torch.log2(want.abs().clamp(min=2.0**-6))) - 3)
    assert bool(((value - want).abs() <= 1.01 * step).all())


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [1e-45, 1e-40, 1.1e-38, 1.2e-38])
def test_an_epsilon_next_to_nothing(eps, bits):
    """Values without a gradient or moments stay where they are; the others step by lr times their sign."""
    p = torch.randn(1000, device="cuda")
    g = torch.randn(1000, device="cuda")
    g[::3] = 0
    q, state = p.clone(), ecc.adamw_state([p], bits)
    ecc.ecc_adamw([q], [g], state, step=1, lr=0.125, weight_decay=0.0, eps=eps)
    # m / sqrt(v) is 1 to 2^-19, the parameter rounds to 2^-24 of at most 8
    assert bool(((p - q) - 0.125 * torch.sign(g)).abs().max() < 2.0**-20) and torch.equal(p[::3], q[::3])
