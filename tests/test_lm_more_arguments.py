"""Argument checks at the C ABI of the gated projections, the log
probabilities of hidden states and AdamW, made before any CUDA call (so they
run without a GPU), and their Python entry points' arguments by name and by
position."""
import ctypes as ct
import math
import struct

import pytest

import lossless_entropy_coding_gb300 as ecc

GATED = struct.Struct("@8P9Q3f6I")            # ecc_gated_linear_job
GATED_GRAD = struct.Struct("@11P12Q2f4I")     # ecc_gated_linear_grad_job
HEAD = struct.Struct("@6P5Qf2I")              # ecc_linear_logprob_job
HEAD_GRAD = struct.Struct("@9P7Qf3I")         # ecc_linear_logprob_grad_job
TENSOR = struct.Struct("@7PQ4I")              # ecc_adamw_tensor
ADAMW = struct.Struct("@PQ6dQ3P2I")           # ecc_adamw_job
P = 1 << 20   # an aligned address that is never read: the calls return before any launch


def gated(status=P, ws=0, ws_bytes=0, **kw):
    a = dict(x=P, w_gate=P, w_up=P, bias_gate=0, bias_up=0, out=2 * P, pre_gate=0, pre_up=0, M=4, N=8, K=16, ldx=16, ldgate=16,
             ldup=16, ldout=8, ldpre_gate=8, ldpre_up=8, scale=1.0, up_scale=1.0, out_scale=1.0, in_type=ecc.BF16,
             bias_type=ecc.F32, out_type=ecc.BF16, pre_type=ecc.BF16, act=4, reserved=0)
    assert not set(kw) - set(a)
    a.update(kw)
    return ecc.lib().ecc_gated_linear(GATED.pack(*a.values()), ws, ws_bytes, status, 0)


def gated_grad(status=P, ws=0, ws_bytes=0, **kw):
    a = dict(dy=P, x=P, w_gate=P, w_up=P, pre_gate=P, pre_up=P, dx=2 * P, dw_gate=2 * P, dw_up=2 * P, dbias_gate=0, dbias_up=0, M=4,
             N=8, K=16, lddy=8, ldx=16, ldgate=16, ldup=16, ldpre_gate=8, ldpre_up=8, lddx=16, lddw_gate=16, lddw_up=16, scale=1.0,
             up_scale=1.0, in_type=ecc.BF16, pre_type=ecc.BF16, dw_type=ecc.BF16, act=4)
    assert not set(kw) - set(a)
    a.update(kw)
    return ecc.lib().ecc_gated_linear_grad(GATED_GRAD.pack(*a.values()), ws, ws_bytes, status, 0)


def head(status=P, ws=0, ws_bytes=0, **kw):
    a = dict(x=P, w=P, tokens=P, logprob=P, entropy=P, lse=P, rows=4, vocab=100, K=16, ldx=16, ldw=16, scale=1.0, in_type=ecc.BF16,
             reserved=0)
    assert not set(kw) - set(a)
    a.update(kw)
    return ecc.lib().ecc_linear_logprob(HEAD.pack(*a.values()), ws, ws_bytes, status, 0)


def head_grad(status=P, ws=0, ws_bytes=0, **kw):
    a = dict(x=P, w=P, tokens=P, lse=P, entropy=P, dlogprob=P, dentropy=P, dx=2 * P, dw=2 * P, rows=4, vocab=100, K=16, ldx=16,
             ldw=16, lddx=16, lddw=16, scale=1.0, in_type=ecc.BF16, dw_type=ecc.BF16, reserved=0)
    assert not set(kw) - set(a)
    a.update(kw)
    return ecc.lib().ecc_linear_logprob_grad(HEAD_GRAD.pack(*a.values()), ws, ws_bytes, status, 0)


def tensor(at=1, **kw):
    a = dict(param=at * 64 * P, grad=P, m=at * 64 * P + 8 * P, v=at * 64 * P + 16 * P, m_scale=0, v_scale=0, master=0, n=1000,
             param_type=ecc.BF16, grad_type=ecc.BF16, state_type=ecc.F32, reserved=0)
    assert not set(kw) - set(a)
    a.update(kw)
    return TENSOR.pack(*a.values())


def adamw(*tensors, **kw):
    data = ct.create_string_buffer(b"".join(tensors), max(1, TENSOR.size * len(tensors)))
    a = dict(tensors=ct.addressof(data), count=len(tensors), lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1,
             grad_scale=1.0, step=1, step_at=0, lr_at=0, grad_scale_at=0, seed=0, reserved=0)
    assert not set(kw) - set(a)
    a.update(kw)
    return ecc.lib().ecc_adamw(ADAMW.pack(*a.values()), 0)


def refused(call, cases):
    for kw in cases:
        assert call(**kw) == ecc.ERR_ARG, kw


def test_gated_refusals():
    refused(gated, [dict(status=0), dict(status=P + 2), dict(x=0), dict(w_gate=0), dict(w_up=0), dict(out=0), dict(x=P + 1),
                    dict(w_up=P + 1), dict(out=P + 1), dict(ldx=15), dict(ldgate=15), dict(ldup=15), dict(ldout=7), dict(in_type=ecc.F32),
                    dict(in_type=9), dict(out_type=9), dict(act=5), dict(scale=math.nan), dict(up_scale=math.inf),
                    dict(out_scale=2.0), dict(M=1 << 31), dict(N=1 << 31), dict(K=1 << 31), dict(bias_gate=P, bias_type=ecc.E4M3),
                    dict(bias_up=P + 2), dict(pre_gate=P), dict(pre_up=P), dict(pre_gate=P, pre_up=P, pre_type=ecc.E4M3),
                    dict(pre_gate=P, pre_up=P, ldpre_up=7), dict(pre_gate=P + 1, pre_up=P), dict(reserved=1)])
    # an operand that has to be copied, without the scratch for it
    refused(gated, [dict(M=100, N=3000, K=1001, ldx=1001, ldgate=1001, ldup=1001, ldout=3000, **w)
                    for w in (dict(), dict(ws=P, ws_bytes=16), dict(ws=P + 8, ws_bytes=1 << 30))])
    assert ecc.lib().ecc_gated_linear(None, 0, 0, P, 0) == ecc.ERR_ARG
    assert ecc.lib().ecc_gated_linear_workspace_bytes(None) == 0


def test_gated_grad_refusals():
    ok = dict(ws=P, ws_bytes=1 << 30)
    refused(gated_grad, [dict(ok, **kw) for kw in (
        dict(status=0), dict(dy=0), dict(x=0), dict(w_gate=0), dict(w_up=0), dict(pre_gate=0), dict(pre_up=0), dict(dy=P + 1),
        dict(dw_up=0), dict(dw_gate=0), dict(dbias_gate=P), dict(dbias_up=P), dict(dbias_gate=P + 2, dbias_up=P), dict(lddy=7),
        dict(ldx=15), dict(ldgate=15), dict(ldup=15), dict(ldpre_gate=7), dict(ldpre_up=7), dict(lddx=15), dict(lddw_gate=15),
        dict(lddw_up=15), dict(in_type=ecc.E4M3), dict(in_type=ecc.F32), dict(pre_type=ecc.E4M3), dict(dw_type=ecc.F16),
        dict(act=5), dict(scale=math.inf), dict(up_scale=math.nan), dict(M=1 << 31))])
    refused(gated_grad, [dict(), dict(ws=P, ws_bytes=64), dict(ws=P + 8, ws_bytes=1 << 30)])
    assert ecc.lib().ecc_gated_linear_grad(None, P, 1 << 30, P, 0) == ecc.ERR_ARG


def test_head_refusals():
    refused(head, [dict(status=0), dict(x=0), dict(w=0), dict(x=P + 1), dict(w=P + 1), dict(tokens=P + 4), dict(logprob=P + 2),
                   dict(entropy=P + 2), dict(lse=P + 2), dict(vocab=0), dict(vocab=1 << 31), dict(rows=1 << 31), dict(K=1 << 31),
                   dict(ldx=15), dict(ldw=15), dict(in_type=ecc.F32), dict(in_type=9), dict(scale=math.nan), dict(reserved=1)])
    ok = dict(ws=P, ws_bytes=1 << 30)
    refused(head_grad, [dict(ok, **kw) for kw in (
        dict(status=0), dict(x=0), dict(w=0), dict(lse=0), dict(entropy=0), dict(lse=P + 2), dict(entropy=P + 1), dict(dlogprob=P + 2),
        dict(dentropy=P + 2), dict(tokens=P + 4), dict(dx=P + 1), dict(dw=P + 1), dict(lddx=15), dict(lddw=15), dict(ldx=15),
        dict(ldw=15), dict(vocab=0), dict(vocab=1 << 31), dict(in_type=ecc.E4M3), dict(dw_type=ecc.F16), dict(scale=math.inf),
        dict(reserved=1))])
    refused(head_grad, [dict(), dict(ws=P, ws_bytes=64), dict(ws=P + 8, ws_bytes=1 << 30)])
    assert ecc.lib().ecc_linear_logprob(None, P, 1 << 30, P, 0) == ecc.ERR_ARG
    assert ecc.lib().ecc_linear_logprob_grad(None, P, 1 << 30, P, 0) == ecc.ERR_ARG


def test_head_grad_workspace_is_bounded():
    def need(rows, vocab, K=64, dx=P):
        a = (P, P, P, P, P, P, P, dx, P, rows, vocab, K, K, K, K, K, 1.0, ecc.BF16, ecc.BF16, 0)
        return ecc.lib().ecc_linear_logprob_grad_workspace_bytes(HEAD_GRAD.pack(*a))

    assert need(4, 1000) < 1 << 16
    # t of a piece: 256 MiB at most; dx's sum beside it
    for rows, vocab in ((4096, 131072), (8192, 262144), (100000, 50021)):
        assert need(rows, vocab) <= (256 << 20) + rows * 64 * 4 + 8192 and need(rows, vocab, dx=0) <= (256 << 20) + 8192
    assert need(1 << 20, 1000) <= (512 << 20) + (1 << 28) + 8192           # 256 tokens of the vocabulary at least


def test_adamw_refusals():
    def call(**kw):
        job = {k: kw.pop(k) for k in list(kw) if k in ("lr", "beta1", "beta2", "eps", "weight_decay", "grad_scale", "step", "step_at",
                                                        "lr_at", "grad_scale_at", "reserved_job")}
        if "reserved_job" in job:
            job["reserved"] = job.pop("reserved_job")
        return adamw(tensor(**kw), **job)

    bytes_ = dict(state_type=ecc.E4M3, m_scale=400 * P, v_scale=401 * P)
    refused(call, [dict(param=0), dict(grad=0), dict(m=0), dict(v=0), dict(param=P + 1), dict(grad=P + 1), dict(m=64 * P + 2),
                   dict(v=64 * P + 2), dict(master=P + 2), dict(n=1 << 40), dict(param_type=ecc.E4M3), dict(grad_type=ecc.E4M3),
                   dict(state_type=ecc.BF16), dict(state_type=ecc.E4M3), dict(bytes_, v_scale=0), dict(bytes_, m_scale=400 * P + 1),
                   dict(reserved=1), dict(reserved_job=1), dict(lr=math.nan), dict(beta1=1.0), dict(beta1=-0.5), dict(beta2=1.0),
                   dict(beta2=math.nan), dict(eps=-1.0), dict(eps=math.inf), dict(weight_decay=math.inf), dict(grad_scale=math.nan),
                   dict(step=0), dict(step=0, step_at=P + 4), dict(lr_at=P + 1), dict(grad_scale_at=P + 2)])
    # arrays that are written and overlap: the same tensor twice, moments in one place, a master in its parameter
    assert adamw(tensor(), tensor()) == ecc.ERR_ARG
    assert adamw(tensor(), tensor(2, v=64 * P + 8 * P + 3996)) == ecc.ERR_ARG
    assert adamw(tensor(v=64 * P + 8 * P)) == ecc.ERR_ARG and adamw(tensor(master=64 * P)) == ecc.ERR_ARG
    assert adamw(tensor(**bytes_), tensor(2, state_type=ecc.E4M3, m_scale=400 * P + 12, v_scale=402 * P)) == ecc.ERR_ARG
    assert ecc.lib().ecc_adamw(None, 0) == ecc.ERR_ARG


def test_adamw_of_nothing_is_accepted():
    assert adamw() == ecc.OK and adamw(tensor(n=0), tensor(n=0)) == ecc.OK


def test_python_entry_points_take_arguments_by_name_and_by_position():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 8)
    calls = {"ecc_gated_linear": dict(x=x, w_gate=x, w_up=x),
             "ecc_gated_linear_grad": dict(dy=x, x=x, w_gate=x, w_up=x, pre_gate=x, pre_up=x),
             "ecc_linear_logprob": dict(x=x, w=x, tokens=None),
             "ecc_linear_logprob_grad": dict(x=x, w=x, tokens=None, lse=x[:, 0]),
             "ecc_adamw": dict(params=[x], grads=[x], state=ecc.AdamWState([x], [x]), step=1)}
    for name, args in calls.items():
        f = getattr(ecc, name)
        for n in range(len(args) + 1):        # the first n by position; a host tensor is refused
            with pytest.raises(ecc.EccError) as e:
                f(*list(args.values())[:n], **dict(list(args.items())[n:]))
            assert e.value.code == ecc.ERR_ARG
        with pytest.raises(TypeError):
            f()
        with pytest.raises(TypeError):
            f(**args, other=1)
    for bad in (dict(params=x), dict(grads=x), dict(state=ecc.AdamWState(x, [x])), dict(state=ecc.AdamWState([x], None))):
        with pytest.raises(ecc.EccError):
            ecc.ecc_adamw(**dict(calls["ecc_adamw"], **bad))
    with pytest.raises(ecc.EccError):
        ecc.adamw_state([x], bits=16)
    state = ecc.adamw_state([x, x.to(torch.bfloat16)], 8, master=True)
    assert [s.shape for s in state.m_scale] == [(1,), (1,)] and state.master[0] is None and state.master[1].dtype == torch.float32
