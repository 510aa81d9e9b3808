"""The random bits of AdamW's 8-bit states are those of a value's place, the
seed and the step, as the header says: tensors of one call share them, calls
with other seeds or steps do not."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import lossless_entropy_coding_gb300 as ecc  # noqa: E402
import test_gpu_adamw as adamw  # noqa: E402

BF16, BYTE, G = torch.bfloat16, torch.uint8, ecc.ADAMW_GROUP


def test_tensors_of_one_call_share_their_random_bits():
    n = 20 * G + 50
    sets = [adamw.make(n, BF16, BF16, 8, False, seed=1) for _ in range(3)]
    state = ecc.AdamWState(*([s[i][0] for _, _, s in sets] for i in range(4)))
    ecc.ecc_adamw([p for p, _, _ in sets], [g for _, g, _ in sets], state, step=3, seed=7)
    for i in (1, 2):
        assert torch.equal(state.m[i], state.m[0]) and torch.equal(state.v[i], state.v[0])
    for seed, step in ((8, 3), (7, 4)):
        p, g, other = adamw.make(n, BF16, BF16, 8, False, seed=1)
        ecc.ecc_adamw([p], [g], other, step=step, seed=seed)
        # a fifth of the codes and more are decided by other bits
        assert int((other.m[0] != state.m[0]).sum()) > n // 5 and int((other.v[0] != state.v[0]).sum()) > n // 5


def test_more_float32_values_than_32_bits_count():
    """(test_gpu_adamw's case of both kinds of states leaves the float32 one out where there is no room: visibly here)"""
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB of free device memory")
    big, tail = 1 << 32, 1000
    p0, g0, s0 = adamw.make(tail, BF16, BF16, 32, False)
    p, g = (torch.zeros(big + tail, dtype=BF16, device="cuda") for _ in range(2))
    state = ecc.adamw_state([p], 32)
    ends = [slice(0, tail), slice(big, big + tail)]
    for e in ends:
        p[e], g[e], state.m[0][e], state.v[0][e] = p0, g0, s0.m[0], s0.v[0]
    ecc.ecc_adamw([p], [g], state, step=3, seed=5, **adamw.HYPER)
    for e in ends:
        adamw.check(p[e], ecc.AdamWState([state.m[0][e]], [state.v[0][e]]), p0, g0, s0, 3, seed=5, **adamw.HYPER)
    assert not p[tail:big].any()
