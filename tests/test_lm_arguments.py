"""Argument checks of the language-model operators at the C ABI, which are made
before any CUDA call (so they run without a GPU): every refusal is ECC_ERR_ARG
and calls over no rows are accepted."""
import ctypes as ct
import math
import struct

import lossless_entropy_coding_gb300 as ecc

LINEAR_JOB = struct.Struct("@6P8Q2f6I")        # ecc_linear_job
LINEAR_GRAD_JOB = struct.Struct("@7P9Qf5I")    # ecc_linear_grad_job
P = 1 << 20   # an aligned address that is never read: the calls return before any launch


def norm(**kw):
    a = dict(x=P, ldx=64, x_type=ecc.BF16, weight=0, bias=0, p_type=ecc.BF16, rows=4, cols=64, eps=1e-5, y=2 * P, ldy=64,
             y_type=ecc.BF16, y_scale=1.0, mean=0, rstd=0, stream=0)
    a.update(kw)
    return ecc.lib().ecc_layer_norm(*a.values())


def norm_grad(**kw):
    a = dict(dy=P, lddy=64, x=P, ldx=64, type=ecc.F16, weight=0, p_type=ecc.F16, mean=P, rstd=P, rows=4, cols=64, dx=2 * P,
             lddx=64, dweight=P, dbias=P, ws=P, ws_bytes=1 << 20, stream=0)
    a.update(kw)
    return ecc.lib().ecc_layer_norm_grad(*a.values())


def logprob(**kw):
    a = dict(logits=P, ld=100, type=ecc.F32, tokens=P, rows=3, vocab=100, scale=1.0, top=2, logprob=P, entropy=P, lse=P,
             top_logprob=P, top_index=P, stream=0)
    a.update(kw)
    return ecc.lib().ecc_token_logprob(*a.values())


def logprob_grad(**kw):
    a = dict(logits=P, ld=100, type=ecc.F32, tokens=P, rows=3, vocab=100, scale=1.0, lse=P, entropy=P, dlogprob=P,
             dentropy=P, dlogits=2 * P, ldd=100, stream=0)
    a.update(kw)
    return ecc.lib().ecc_token_logprob_grad(*a.values())


def linear(status=P, ws=0, ws_bytes=0, **kw):
    a = dict(x=P, w=P, bias=0, residual=0, out=2 * P, pre=0, M=4, N=8, K=16, ldx=16, ldw=16, ldres=8, ldout=8, ldpre=8,
             scale=1.0, out_scale=1.0, in_type=ecc.BF16, bias_type=ecc.F32, res_type=ecc.F32, out_type=ecc.BF16,
             pre_type=ecc.BF16, act=0)
    a.update(kw)
    return ecc.lib().ecc_linear(LINEAR_JOB.pack(*a.values()), ws, ws_bytes, status, 0)


def linear_grad(status=P, ws=0, ws_bytes=0, **kw):
    a = dict(dy=P, x=P, w=P, pre=0, dx=2 * P, dw=2 * P, dbias=0, M=4, N=8, K=16, lddy=8, ldx=16, ldw=16, ldpre=8,
             lddx=16, lddw=16, scale=1.0, in_type=ecc.BF16, pre_type=ecc.BF16, dw_type=ecc.BF16, act=0, reserved=0)
    a.update(kw)
    return ecc.lib().ecc_linear_grad(LINEAR_GRAD_JOB.pack(*a.values()), ws, ws_bytes, status, 0)


def refused(call, cases):
    for kw in cases:
        assert call(**kw) == ecc.ERR_ARG, kw


def test_layer_norm_arguments():
    refused(norm, [dict(cols=0), dict(x=0), dict(y=0), dict(ldx=63), dict(ldy=63), dict(x=P + 1), dict(x_type=ecc.E4M3),
                   dict(x_type=7), dict(y_type=ecc.F32), dict(p_type=ecc.F16), dict(weight=P + 2, p_type=ecc.F32),
                   dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(y_scale=2.0),
                   dict(y_type=ecc.E4M3, y_scale=math.nan), dict(mean=P + 2), dict(x=2 * P, ldx=72), dict(cols=1 << 31)])
    assert norm(rows=0, x=0, y=0) == ecc.OK
    refused(norm_grad, [dict(cols=0), dict(dy=0), dict(x=0), dict(mean=0), dict(rstd=0), dict(lddy=63), dict(ldx=63),
                        dict(lddx=63), dict(type=ecc.E4M3), dict(p_type=ecc.BF16), dict(ws=0), dict(ws=P + 8),
                        dict(ws_bytes=15), dict(dx=P, lddx=72), dict(dweight=P + 1)])
    assert norm_grad(rows=0, dweight=0, dbias=0, ws=0) == ecc.OK


def test_token_logprob_arguments():
    refused(logprob, [dict(vocab=0), dict(vocab=1 << 31), dict(logits=0), dict(ld=99), dict(type=ecc.E4M3), dict(top=33),
                      dict(vocab=1, top=2), dict(top_index=0), dict(scale=0.0), dict(scale=math.nan), dict(tokens=P + 4),
                      dict(logits=P + 2), dict(lse=P + 2)])
    assert logprob(rows=0, logits=0) == ecc.OK
    refused(logprob_grad, [dict(vocab=0), dict(logits=0), dict(dlogits=0), dict(lse=0), dict(ld=99), dict(ldd=99),
                           dict(tokens=0), dict(entropy=0), dict(scale=-1.0), dict(dlogits=P, ldd=104),
                           dict(type=ecc.E4M3)])
    assert logprob_grad(rows=0) == ecc.OK


def test_linear_arguments():
    refused(linear, [dict(status=0), dict(status=P + 2), dict(x=0), dict(w=0), dict(out=0), dict(ldx=15), dict(ldw=15),
                     dict(ldout=7), dict(x=P + 1), dict(in_type=ecc.F32), dict(in_type=9), dict(out_type=9), dict(act=5),
                     dict(bias=P, bias_type=ecc.E4M3), dict(residual=P, ldres=7), dict(residual=P, res_type=ecc.E4M3),
                     dict(residual=2 * P, ldres=9, res_type=ecc.BF16), dict(pre=P, ldpre=7),
                     dict(pre=P, pre_type=ecc.E4M3), dict(scale=math.inf), dict(out_scale=0.5), dict(M=1 << 31),
                     dict(K=1 << 31, ldx=1 << 31, ldw=1 << 31)])
    refused(linear_grad, [dict(status=0), dict(dy=0), dict(x=0), dict(w=0), dict(lddy=7), dict(ldx=15), dict(ldw=15),
                          dict(lddx=15), dict(lddw=15), dict(in_type=ecc.E4M3), dict(in_type=ecc.F32),
                          dict(dw_type=ecc.F16), dict(act=2), dict(act=5), dict(act=2, pre=P), dict(dbias=P + 2),
                          dict(scale=math.nan)])
    assert ecc.lib().ecc_linear(None, 0, 0, P, 0) == ecc.ERR_ARG
    assert ecc.lib().ecc_linear_grad(None, 0, 0, P, 0) == ecc.ERR_ARG
    assert struct_sizes() == (144, 152)


def struct_sizes():
    return LINEAR_JOB.size, LINEAR_GRAD_JOB.size


def test_workspace_sizes_need_no_gpu():
    lib = ecc.lib()
    assert lib.ecc_layer_norm_grad_workspace_bytes(0, 64) >= 0
    assert lib.ecc_layer_norm_grad_workspace_bytes(1 << 20, 64) >= 64 * 8
    assert isinstance(ct.c_size_t(lib.ecc_linear_workspace_bytes(None)).value, int)
