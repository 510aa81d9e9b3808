"""AdamW over many tensors against the formula in 64 bits: types, masters,
8-bit states with their dithered rounding, unaligned and empty tensors, steps
read from the device, captured calls, refusals.

Tolerances: float32 moments are two products and a sum, each rounded by at
most 2^-24 of the summands, with coefficients rounded once: 2^-22 of the
summands' magnitudes.  The parameter's update divides them (quotient, root and
reciprocal of 2^-22 each): 2^-19 of rate * summands / denominator, plus 2^-22
of the parameter, plus half a step of its type.  The value an 8-bit state is
rounded from is off by the moment's 2^-22 of its summands (which may cancel)
and by 2^-21 of itself from the scale: the dither's threshold, of 65536 steps,
moves by as much of the distance of its two e4m3 neighbours, and by one for
the bits that the addition drops."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import lossless_entropy_coding_gb300 as ecc  # noqa: E402

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
E4M3, BYTE, G = torch.float8_e4m3fn, torch.uint8, ecc.ADAMW_GROUP
HYPER = dict(lr=2e-3, beta1=0.9, beta2=0.95, eps=1e-6, weight_decay=0.1)


def mix(x):
    m = 0xFFFFFFFF
    x = x ^ (x >> 16)
    x = (x * 0x7FEB352D) & m
    x = x ^ (x >> 15)
    x = (x * 0x846CA68B) & m
    return x ^ (x >> 16)


def random_bits(n, seed, step, high=0):
    key = mix(torch.tensor((int(mix(torch.tensor(seed))) + step) & 0xFFFFFFFF))
    bits = mix(torch.arange(n) ^ int(mix((key + high) & 0xFFFFFFFF))).cuda()
    return bits >> 16, bits & 0xFFFF


def coded(value, size, bits, positive=False):
    """(e4m3 value, scale, whether the dither is clear of its threshold) of 64-bit values."""
    n = value.numel()
    pad = torch.zeros(-(-n // G) * G, dtype=torch.float64, device=value.device)
    pad[:n] = value.abs()
    scale = pad.view(-1, G).amax(-1) / 448
    each = scale.repeat_interleave(G)[:n]
    a = torch.where(each > 0, value.abs() / each, 0).clamp(max=448)
    ulp = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0**-6))) - 3)
    low = torch.floor(a / ulp)
    reach = (a / ulp - low) * 65536 + bits
    c = (low + (reach >= 65536)) * ulp
    if positive:
        c = torch.where(value > 0, c.clamp(min=2.0**-9), 0)
    off = torch.where(each > 0, (2.0**-22 * size + 2.0**-21 * value.abs()) / each, 0) / ulp
    edge = (a / ulp - torch.round(a / ulp)).abs() <= off         # its neighbours themselves may differ
    return torch.sign(value) * c, scale, ((reach - 65536).abs() > 1 + 65536 * off) & ~edge


def make(n, ptype, gtype, bits, master, seed=0, skew=0):
    g = torch.Generator("cuda").manual_seed(seed + n)

    def normal(std=1.0, dtype=F32):
        t = torch.empty(n + 64, dtype=dtype, device="cuda")[skew:skew + n]
        return t.copy_(torch.randn(n, generator=g, device="cuda") * std)

    p = normal(0.05, ptype)
    state = ecc.adamw_state([p], bits, master)
    if bits == 8:
        m, v = (torch.empty(n + 64, dtype=BYTE, device="cuda")[skew:skew + n] for _ in range(2))
        m.copy_(normal(100).clamp(-448, 448).to(E4M3).view(BYTE))
        v.copy_(normal(100).abs().clamp(max=448).to(E4M3).view(BYTE))
        state.m_scale[0].copy_(torch.rand(-(-n // G), generator=g, device="cuda") * 1e-4)
        state.v_scale[0].copy_(torch.rand(-(-n // G), generator=g, device="cuda") * 1e-3)
        state = state._replace(m=[m], v=[v])
    else:
        state = state._replace(m=[normal(0.01)], v=[normal(0.03).square_()])
    return p, normal(0.02, gtype), state


def reference(p, grad, state, step, grad_scale=1.0, lr=None, beta1=0.9, beta2=0.95, eps=0.0, weight_decay=0.0):
    """64-bit moments, parameter, and the magnitudes their errors are measured by."""
    n = p.numel()
    m, v = state.m[0], state.v[0]
    if state.m_scale is not None:
        ms, vs = (s[0].double().repeat_interleave(G)[:n] for s in (state.m_scale, state.v_scale))
        m, v = m.view(E4M3).double() * ms, (v.view(E4M3).double() * vs)**2
    m, v, g = m.double(), v.double(), grad.double() * grad_scale
    f = (p if state.master is None or state.master[0] is None else state.master[0]).double()
    size = beta1 * m.abs() + (1 - beta1) * g.abs()
    m, v = beta1 * m + (1 - beta1) * g, beta2 * v + (1 - beta2) * g * g
    rate, den = lr / (1 - beta1**step), (v / (1 - beta2**step)).sqrt() + eps
    return m, v, f * (1 - lr * weight_decay) - rate * m / den, size, f.abs() * 2.0**-22 + rate * size / den * 2.0**-19


def copied(state):
    return ecc.AdamWState(*([t.clone() if t is not None else None for t in x] if x is not None else None for x in state))


def check(p, state, old_p, grad, old, step, seed=0, high=0, **hyper):
    m, v, f, size, slack = reference(old_p, grad, old, step, **hyper)
    half = torch.finfo(p.dtype).eps / 2
    tiny = torch.finfo(p.dtype).smallest_normal * torch.finfo(p.dtype).eps / 2   # half a step of subnormals
    assert ((p.double() - f).abs() <= slack + half * f.abs() * (1 + half) + tiny).all()
    if state.master is not None and state.master[0] is not None:
        assert ((state.master[0].double() - f).abs() <= slack + 2.0**-24 * f.abs()).all()
    if state.m_scale is None:
        assert ((state.m[0].double() - m).abs() <= 2.0**-22 * size + 1e-44).all()
        assert ((state.v[0].double() - v).abs() <= 2.0**-22 * v + 1e-44).all()
        return
    upper, lower = random_bits(m.numel(), seed, step, high)
    for got, scale, want, size, bits, positive in ((state.m[0], state.m_scale[0], m, size, upper, False),
                                                   (state.v[0], state.v_scale[0], v.sqrt(), v.sqrt(), lower, True)):
        value, s, clear = coded(want, size, bits, positive)
        most = torch.zeros(s.numel() * G, dtype=torch.float64, device="cuda")
        most[:size.numel()] = size
        assert ((scale.double() - s).abs() <= 2.0**-22 * (s + most.view(-1, G).amax(-1) / 448)).all()
        got = got.view(E4M3).double()
        assert torch.equal(got[clear], value[clear])
        step_of = torch.exp2(torch.floor(torch.log2(value.abs().clamp(min=2.0**-6))) - 3) * 1.01
        assert ((got - value).abs() <= step_of).all()


@pytest.mark.parametrize("n", [1, 7, 255, 256, 257, 2048, 5000, 70001])
@pytest.mark.parametrize("ptype,gtype,bits,master", [(F32, F32, 32, False), (BF16, BF16, 32, False), (F16, F32, 32, True),
                                                     (BF16, F32, 32, True), (F32, BF16, 8, False), (BF16, BF16, 8, True),
                                                     (F16, F16, 8, False), (BF16, F16, 8, False)])
def test_one_tensor(n, ptype, gtype, bits, master):
    for skew in (0, 8, 3):
        p, g, state = make(n, ptype, gtype, bits, master, skew=skew)
        old_p, old = p.clone(), copied(state)
        ecc.ecc_adamw([p], [g], state, step=3, seed=5, **HYPER)
        check(p, state, old_p, g, old, 3, seed=5, **HYPER)


def test_many_tensors_of_all_kinds_in_one_call():
    kinds = [(F32, F32, 32, False), (BF16, BF16, 8, True), (F16, F32, 8, False), (BF16, F32, 32, True)]
    items = [make(1 + 97 * i % 5003, *kinds[i % 4], seed=i, skew=i % 3) for i in range(1100)]
    empty = make(256, F32, F32, 32, False)
    items[7] = (empty[0][:0], empty[1][:0], ecc.AdamWState([empty[0][:0]], [empty[0][:0]]))
    state = ecc.AdamWState([s.m[0] for _, _, s in items], [s.v[0] for _, _, s in items],
                           [s.m_scale[0] if s.m_scale else None for _, _, s in items],
                           [s.v_scale[0] if s.v_scale else None for _, _, s in items],
                           [s.master[0] if s.master else None for _, _, s in items])
    grads = [g for _, g, _ in items]
    grads[11] = None                                     # left alone
    old = [(p.clone(), copied(s)) for p, _, s in items]
    ecc.ecc_adamw([p for p, _, _ in items], grads, state, step=20, grad_scale=0.5, **HYPER)
    for i, (p, g, s) in enumerate(items):
        if i == 11:
            assert torch.equal(p, old[i][0]) and torch.equal(s.m[0], old[i][1].m[0])
        elif p.numel():
            check(p, s, old[i][0], g, old[i][1], 20, grad_scale=0.5, **HYPER)


def test_moments_round_as_separate_products_and_sums():
    """To the bit: m beta1, g (1 - beta1), their sum; the 8-bit states follow from those."""
    n = 40000
    p, g, state = make(n, F32, F32, 32, False)
    m, v = state.m[0].clone(), state.v[0].clone()
    ecc.ecc_adamw([p], [g], state, step=5, **HYPER)
    assert torch.equal(state.m[0], m * 0.9 + g * (1 - 0.9))
    assert torch.equal(state.v[0], v * 0.95 + g * g * (1 - 0.95))


@pytest.mark.parametrize("spread", [0.0, 1.0, 6.0, 20.0])
def test_vectors_and_single_values_give_the_same_codes(spread):
    """Groups with and without values below the smallest normal code, at aligned and unaligned addresses."""
    n = 20 * G
    p, g, state = make(n, F32, F32, 8, False, seed=3)
    wide = torch.exp(torch.randn(n, device="cuda") * spread)
    g = g * wide
    state.m[0].view(E4M3)[::5] = 0
    state.v[0].view(E4M3)[::5] = 0
    g[::10] = 0                                          # zero moments among the others
    other = [torch.empty(n + 1, dtype=t.dtype, device="cuda")[1:].copy_(t) for t in (p, g, state.m[0], state.v[0])]
    old_p, old = p.clone(), copied(state)
    s2 = ecc.AdamWState([other[2]], [other[3]], [state.m_scale[0].clone()], [state.v_scale[0].clone()])
    ecc.ecc_adamw([p], [g], state, step=4, **HYPER)
    ecc.ecc_adamw([other[0]], [other[1]], s2, step=4, **HYPER)
    # (0.02 e^(20 * 4.5), the largest of 5120 gradients, has a square of 10^74: no float32 and no such update)
    if float(g.double().square().max()) < 3e38:
        check(p, state, old_p, g, old, 4, **HYPER)
    assert torch.equal(p, other[0]) or bool((p.isnan() == other[0].isnan()).all())
    for a, b in zip(state[:4], s2[:4]):
        assert torch.equal(a[0].view(BYTE), b[0].view(BYTE))
    if bool(torch.isfinite(state.m_scale[0]).all()):
        assert not state.m[0].view(E4M3).float()[::10].any() and not state.v[0][::10].any()


def test_more_values_than_32_bits_count():
    big, tail = 1 << 32, 1000
    for bits in (8, 32):
        if bits == 32 and torch.cuda.mem_get_info()[0] < 80 << 30:
            continue
        p0, g0, s0 = make(tail, BF16, BF16, bits, False)
        p, g = (torch.zeros(big + tail, dtype=BF16, device="cuda") for _ in range(2))
        state = ecc.adamw_state([p], bits)
        ends = [slice(0, tail), slice(big, big + tail)]
        for e in ends:
            p[e], g[e], state.m[0][e], state.v[0][e] = p0, g0, s0.m[0], s0.v[0]
            if bits == 8:
                groups = slice(e.start // G, e.start // G + s0.m_scale[0].numel())
                state.m_scale[0][groups], state.v_scale[0][groups] = s0.m_scale[0], s0.v_scale[0]
        ecc.ecc_adamw([p], [g], state, step=3, seed=5, **HYPER)
        for high, e in enumerate(ends):
            groups = slice(e.start // G, e.start // G + -(-tail // G))
            got = ecc.AdamWState([state.m[0][e]], [state.v[0][e]], *([[x[0][groups]] for x in state[2:4]] if bits == 8 else (None, None)))
            check(p[e], got, p0, g0, s0, 3, seed=5, high=high, **HYPER)
        assert not p[tail:big].any()
        del p, g, state
        torch.cuda.empty_cache()


def test_nothing_beyond_the_tensors_is_written():
    n = 1000
    for bits in (8, 32):
        for skew in (0, 1):
            whole = [torch.full((n + 32,), 7, dtype=t, device="cuda")
                     for t in (BF16, BYTE if bits == 8 else F32, BYTE if bits == 8 else F32)]
            p, m, v = (w[8 + skew:8 + skew + n] for w in whole)
            scales = [torch.ones(6, device="cuda") for _ in range(2)]
            g = torch.ones(n, dtype=BF16, device="cuda")
            s = ecc.AdamWState([m], [v], [scales[0][1:5]], [scales[1][1:5]]) if bits == 8 else ecc.AdamWState([m], [v])
            ecc.ecc_adamw([p], [g], s, step=1)
            for w in whole:
                assert (w[:8 + skew] == 7).all() and (w[8 + skew + n:] == 7).all()
            assert float(scales[0][0]) == 1 and float(scales[0][5]) == 1


def test_steps_from_zero_states_and_the_first_update():
    p = torch.randn(3000, device="cuda")
    g = torch.randn(3000, device="cuda")
    for bits in (32, 8):
        q = p.clone()
        state = ecc.adamw_state([q], bits)
        ecc.ecc_adamw([q], [g], state, step=1, lr=0.1, weight_decay=0.0, eps=0.0)
        # m / sqrt(v) is the sign of the first gradient
        assert ((p - q) - 0.1 * torch.sign(g)).abs().max() < 1e-5


def test_zero_gradients_and_states():
    for bits in (32, 8):
        p = torch.ones(600, device="cuda", dtype=BF16)
        state = ecc.adamw_state([p], bits, master=True)
        ecc.ecc_adamw([p], [torch.zeros_like(p)], state, step=1, weight_decay=0.0)
        assert (p == 1).all() and (state.master[0] == 1).all()
        assert not state.m[0].any() and not state.v[0].any()


def test_dithered_states_keep_small_changes_on_average():
    """A root that each step changes by less than half its neighbours' distance still gets there."""
    n = 1 << 16
    p = torch.zeros(n, device="cuda")
    state = ecc.adamw_state([p], 8)
    g = torch.full((n,), 0.5, device="cuda")
    g[::G] = 1.0                                         # each group's largest
    state.v[0].view(E4M3).fill_(256)                     # roots of 1 (scale 1/256), to become 1/2
    state.v_scale[0].fill_(1 / 256)
    steps = 120
    for t in range(1, steps + 1):
        ecc.ecc_adamw([p], [g], state, step=t, lr=0.0, beta2=0.95, seed=9)
    v = (state.v[0].view(E4M3).float() * state.v_scale[0].repeat_interleave(G)).square()
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    rest[::G] = False
    want = 0.25 + 0.75 * 0.95**steps
    # the dither of a root r adds the variance of r's own error to the mean of r^2 (a step of at most
    # 2^-3 r: at most 2^-8 r^2 each time, kept for 1 / (1 - beta2) = 20 steps: under 8%)
    assert want * 0.99 < float(v[rest].mean()) < want * 1.08


def test_values_that_are_not_finite():
    n = 1024
    for bad in (math.nan, math.inf, -math.inf):
        for bits in (32, 8):
            p = torch.ones(n, device="cuda")
            state = ecc.adamw_state([p], bits)
            g = torch.ones(n, device="cuda")
            g[300] = bad
            ecc.ecc_adamw([p], [g], state, step=1)
            ok = torch.arange(n, device="cuda") != 300
            assert torch.isfinite(p[ok]).all() and not torch.isfinite(p[300])
            if bits == 8:
                assert torch.isnan(state.m_scale[0]).tolist() == [False, True, False, False]
                assert torch.isnan(state.v_scale[0]).tolist() == [False, True, False, False]
            else:
                assert torch.isfinite(state.m[0][ok]).all()


def test_step_rate_and_scale_on_the_device_and_replayed():
    p, g, state = make(5000, BF16, F32, 8, True)
    q, old, s2 = p.clone(), p.clone(), copied(state)
    step = torch.ones(1, dtype=torch.int64, device="cuda")
    lr, gs = torch.tensor([1e-3], device="cuda"), torch.tensor([0.5], device="cuda")
    keep = copied(state)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    args = dict(beta1=0.9, beta2=0.95, eps=1e-6, weight_decay=0.1, seed=1)
    with torch.cuda.graph(graph, stream=stream):
        ecc.ecc_adamw([p], [g], state, step=step, lr=lr, grad_scale=gs, **args)
    p.copy_(old)
    for a, b in zip(state, keep):
        a[0].copy_(b[0])
    for t, rate in ((1, 1e-3), (2, 4e-3), (7, 2e-3)):
        step.fill_(t)
        lr.fill_(rate)
        before, was = p.clone(), copied(state)
        graph.replay()
        check(p, state, before, g, was, t, seed=1, lr=rate, grad_scale=0.5, beta1=0.9, beta2=0.95, eps=1e-6,
              weight_decay=0.1)
        ecc.ecc_adamw([q], [g], s2, step=t, lr=rate, grad_scale=0.5, **args)
        # (the two forms of 1 - beta^t agree to 2^-21: the states to a step of few of them)
        assert (state.m[0] != s2.m[0]).float().mean() < 1e-3


def test_many_tensors_captured_and_replayed():
    """More tensors than a launch's parameters hold, of both kinds of states."""
    items = [make(300 + i, BF16, BF16, 8 if i % 2 else 32, False, seed=i) for i in range(1000)]
    params, grads = [p for p, _, _ in items], [g for _, g, _ in items]
    state = ecc.AdamWState([s.m[0] for _, _, s in items], [s.v[0] for _, _, s in items],
                           [s.m_scale[0] if s.m_scale else None for _, _, s in items],
                           [s.v_scale[0] if s.v_scale else None for _, _, s in items])
    start = [(p.clone(), copied(s)) for p, _, s in items]
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        ecc.ecc_adamw(params, grads, state, step=6, **HYPER)
    graph.replay()
    torch.cuda.synchronize()
    for (p, g, s), (old_p, old) in list(zip(items, start))[::37]:
        check(p, s, old_p, g, old, 6, **HYPER)


def test_the_same_call_gives_the_same_bits_on_another_stream():
    p, g, state = make(30000, BF16, BF16, 8, False)
    q, s2 = p.clone(), copied(state)
    ecc.ecc_adamw([p], [g], state, step=2, **HYPER)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    ecc.ecc_adamw([q], [g], s2, step=2, stream=stream, **HYPER)
    torch.cuda.current_stream().wait_stream(stream)
    assert torch.equal(p, q) and all(torch.equal(a[0], b[0]) for a, b in zip(state[:4], s2[:4]))


def test_states_travel_coded():
    p, g, state = make(1 << 16, BF16, BF16, 8, False)
    ecc.ecc_adamw([p], [g], state, step=2, **HYPER)
    for t in (state.m[0], state.v[0]):
        t = t.clone()
        count = ecc.e4m3_histogram(t)
        cb = ecc.to_device(ecc.huff_build_canonical(count.cpu().numpy().view("uint64") + 1))
        enc = ecc.ecc_encode(t, cb)
        out, status = ecc.ecc_decode(enc, cb)
        assert int(status.item()) == 0 and torch.equal(out[:t.numel()], t)


def test_refusals():
    p, g, state = make(1000, BF16, BF16, 8, False)

    def refused(params=(p,), grads=(g,), st=state, **kw):
        with pytest.raises(ecc.EccError) as e:
            ecc.ecc_adamw(list(params), list(grads), st, **dict(dict(step=1), **kw))
        assert e.value.code == ecc.ERR_ARG

    for kw in (dict(step=0), dict(step=-3), dict(lr=math.nan), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.5),
               dict(eps=-1.0), dict(eps=math.inf), dict(weight_decay=math.nan), dict(grad_scale=math.inf), dict(seed=-1),
               dict(seed=1 << 32), dict(step=torch.ones(1, device="cuda")), dict(step=torch.ones(2, dtype=torch.int64, device="cuda")),
               dict(lr=torch.ones(1, device="cuda", dtype=torch.float64)), dict(step=torch.ones(1, dtype=torch.int64))):
        refused(**kw)
    refused(grads=(g[:-1],))
    refused(grads=(g.to(torch.float64),))
    refused(params=(p.to(torch.int32),))
    refused(params=(p.cpu(),))
    refused(grads=(torch.stack([g, g], 1)[:, 0],))
    refused(st=ecc.AdamWState(state.m, state.v))
    refused(st=state._replace(m=[state.m[0][:-1]]))
    refused(st=state._replace(v=[state.v[0].to(F32)]))
    refused(st=state._replace(m_scale=[state.m_scale[0][:-1]]))
    refused(st=state._replace(master=[p]))
    refused(st=state._replace(m=state.m * 2))
    twice = ecc.AdamWState(*(x * 2 if x is not None else None for x in state))
    refused(params=(p, p), grads=(g, g), st=twice)       # the same tensor twice
    refused(st=state._replace(v=state.m))
    before = p.clone()
    assert ecc.ecc_adamw([], [], ecc.AdamWState([], []), step=1) is None
    assert torch.equal(p, before)
