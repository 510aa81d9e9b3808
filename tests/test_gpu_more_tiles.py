"""The persistent kernels of the gated projections and of the head with more
tiles than CTAs: accumulators taken in turns, segments of the reduction,
ragged last tiles, results through shared memory, both outputs of one product.
The comparisons and their tolerances are those of the operators' own tests."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import lossless_entropy_coding_gb300 as ecc  # noqa: E402
import test_gpu_gated as gated  # noqa: E402
import test_gpu_head as head  # noqa: E402
import test_gpu_linear as linear  # noqa: E402

F32, BF16, F16, E4M3 = torch.float32, torch.bfloat16, torch.float16, torch.float8_e4m3fn


@pytest.mark.parametrize("dtype", [BF16, F16, E4M3])
@pytest.mark.parametrize("M,N,K,pad", [(2100, 4000, 520, 0), (4096, 2816, 192, 3), (1500, 5001, 264, 0)])
def test_gated_tiles(M, N, K, pad, dtype):
    gen = torch.Generator("cuda").manual_seed(M + N)
    x, wg, wu = (gated.rows_of(gen, r, K, dtype, pad) for r in (M, N, N))
    bg, bu = gated.rows_of(gen, 2, N, F32)
    gated.check(x, wg, wu, bg, bu, "gelu", 1 / math.sqrt(K), pre_dtype=BF16, pre_pad=5)
    gated.check(x, wu, wg, None, None, "silu", 1 / math.sqrt(K), out_dtype=E4M3, out_scale=8.0)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M,N,K,pad", [(2100, 3008, 1024, 0), (900, 4001, 2056, 0), (1111, 2500, 1030, 3), (300, 9000, 2304, 0)])
def test_gated_grad_tiles(M, N, K, pad, dtype):
    gen = torch.Generator("cuda").manual_seed(M + N)
    x, wg, wu = (gated.rows_of(gen, r, K, dtype, pad, std=s) for r, s in ((M, 1.0), (N, N**-0.5), (N, N**-0.5)))
    dy, g, u = (gated.rows_of(gen, M, N, dtype, pad) for _ in range(3))
    a = gated.check_grad(dy, x, wg, wu, g, u, "silu", 1.0, 0.5)
    b = gated.check_grad(dy, x, wg, wu, g, u, "silu", 1.0, 0.5, dw_dtype=F32)
    assert torch.equal(a[0], b[0]) and all(torch.equal(p, q.to(dtype)) for p, q in zip(a[1:3], b[1:3]))


@pytest.mark.parametrize("out_dtype", [BF16, F16, F32])
@pytest.mark.parametrize("M,N,K", [(2300, 4104, 64), (5000, 3000, 200), (1030, 8200, 1024)])
def test_short_reductions_through_shared_memory(M, N, K, out_dtype):
    gen = torch.Generator("cuda").manual_seed(M + N)
    x, w, bias = linear.rows_of(gen, M, K, BF16), linear.rows_of(gen, N, K, BF16), linear.rows_of(gen, 1, N, F32)[0]
    plain = linear.check(x, w, bias, None, "gelu", 1 / math.sqrt(K), out_dtype)
    # into rows that the copies cannot take, and into wider ones: the same values, nothing beside them
    for pad, off in ((1, 1), (8, 8)):
        whole = torch.full((M + 2, N + 2 * pad + 8), 7.0, dtype=out_dtype, device="cuda")
        out = whole[1:M + 1, off:off + N]
        ecc.ecc_linear(x, w, bias, act="gelu", scale=1 / math.sqrt(K), out=out)
        assert torch.equal(out, plain)
        out.fill_(7)
        assert bool((whole == 7).all())


@pytest.mark.parametrize("out_dtype,pre_dtype", [(BF16, BF16), (F32, F16), (E4M3, BF16), (F16, F32), (F32, F32)])
@pytest.mark.parametrize("M,N,K", [(2300, 4112, 64), (4000, 2504, 712)])
def test_gated_short_reductions_through_shared_memory(M, N, K, out_dtype, pre_dtype):
    gen = torch.Generator("cuda").manual_seed(M + N)
    x, wg, wu = (gated.rows_of(gen, r, K, BF16) for r in (M, N, N))
    bg, bu = gated.rows_of(gen, 2, N, F32)
    s = 1 / math.sqrt(K)
    out_scale = 8.0 if out_dtype == E4M3 else 1.0
    for a, b in ((wg, wu), (wu, wg)):
        plain = gated.check(x, a, b, bg, bu, "silu", s, out_dtype=out_dtype, out_scale=out_scale, pre_dtype=pre_dtype)
        results = []
        for pad in (16, 1):                              # rows that the copies can take, and that they cannot
            whole = [torch.full((M + 2, N + 2 * pad + 16), 7.0, device="cuda").to(t) for t in (out_dtype, pre_dtype, pre_dtype)]
            out, g, u = (t[1:M + 1, pad:N + pad] for t in whole)
            ecc.ecc_gated_linear(x, a, b, bg, bu, act="silu", scale=s, out=out, out_scale=out_scale, pre_gate=g, pre_up=u)
            assert torch.equal(out.float(), plain.float())
            results.append((g.clone(), u.clone()))
            for t, v in zip(whole, (out, g, u)):
                v.copy_(torch.full((M, N), 7.0, device="cuda").to(t.dtype))
                assert bool((t.float() == 7).all())
        assert all(torch.equal(p, q) for p, q in zip(*results))


def test_gradients_through_shared_memory_stay_in_their_rows():
    gen = torch.Generator("cuda").manual_seed(5)
    for M, N, K in ((64, 9001, 4096), (200, 8200, 2048)):
        x, wg, wu = gated.rows_of(gen, M, K, BF16), gated.rows_of(gen, N, K, BF16, std=0.01), gated.rows_of(gen, N, K, BF16, std=0.01)
        dy, g, u = (gated.rows_of(gen, M, N, BF16) for _ in range(3))
        for dtype in (BF16, F32):
            whole = [torch.full((N + 2, K + 16), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
            views = [t[1:N + 1, 8:K + 8] for t in whole]
            gated.check_grad(dy, x, wg, wu, g, u, dw_gate=views[0], dw_up=views[1])
            for t, v in zip(whole, views):
                v.fill_(7)
                assert bool((t == 7).all())


# rows, vocab, K: streamed past few tokens, or in pairs; several segments of the reduction
HEADS = [(3, 30001, 1100), (16, 20000, 2050), (40, 40000, 600), (64, 25000, 3000), (65, 20100, 1300), (600, 12000, 1300), (1030, 9001, 600)]


@pytest.mark.parametrize("dtype", [BF16, F16, E4M3])
@pytest.mark.parametrize("M,V,K", HEADS)
def test_head_tiles(M, V, K, dtype):
    gen = torch.Generator("cuda").manual_seed(M + V)
    x, w = head.rows_of(gen, M, K, dtype), head.rows_of(gen, V, K, dtype)
    tok = head.tokens_of(gen, M, V)
    tok[:2] = torch.tensor([0, V - 1])
    first = head.check(x, w, tok, 2 / math.sqrt(K))
    again = ecc.ecc_linear_logprob(x, w, tok, scale=2 / math.sqrt(K))
    assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M,V,K", HEADS)
def test_head_grad_tiles(M, V, K, dtype):
    gen = torch.Generator("cuda").manual_seed(M + V)
    x, w, tok = head.rows_of(gen, M, K, dtype), head.rows_of(gen, V, K, dtype, std=K**-0.5), head.tokens_of(gen, M, V)
    head.check_grad(x, w, tok, 1.5, torch.randn(M, generator=gen, device="cuda"), torch.randn(M, generator=gen, device="cuda") * 0.1)


def test_logits_sums_do_not_lose_what_a_long_accumulation_does():
    """lse of 8192 products a logit to 2^-20 of itself: float32 additions of 16 segments, 512 truncated ones in each."""
    gen = torch.Generator("cuda").manual_seed(7)
    for M in (5, 300):
        x, w = head.rows_of(gen, M, 8192, BF16), head.rows_of(gen, 20480, 8192, BF16, std=2.5 / math.sqrt(8192))
        r = ecc.ecc_linear_logprob(x, w)
        lse = torch.logsumexp(x.double() @ w.double().T, -1)
        # logits near the largest, about 12, of sums that pass through 12 / 16 a segment: 32 steps of 16 products,
        # each short by at most 2^-23 of that, 16 times over: 2^-18 at the most, half of it on average
        assert float(((r.lse.double() - lse) / lse).abs().max()) < 2.0**-18
        assert float(((r.lse.double() - lse) / lse).mean().abs()) < 2.0**-19


def test_captured_calls_that_share_a_workspace():
    """Two graphs over one workspace and status, replayed in turns: each leaves its own results."""
    gen = torch.Generator("cuda").manual_seed(9)
    ws = torch.empty(600 << 20, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cases = []
    for M, V, K in ((500, 30000, 640), (24, 40000, 1100)):
        x, w, tok = head.rows_of(gen, M, K, F16), head.rows_of(gen, V, K, F16, std=0.1), head.tokens_of(gen, M, V)
        dlp = torch.randn(M, generator=gen, device="cuda")
        args = (x, w, tok, dlp)
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=stream):
            r = ecc.ecc_linear_logprob(x, w, tok, ws=ws, status=status)
            g = ecc.ecc_linear_logprob_grad(x, w, tok, r.lse, None, dlp, ws=ws, status=status)
        cases.append((args, graph, r, g))
    for _ in range(3):
        for (x, w, tok, dlp), graph, r, g in cases:
            x.copy_(torch.randn(x.shape, generator=gen, device="cuda"))
            graph.replay()
        torch.cuda.synchronize()
        for (x, w, tok, dlp), graph, r, g in cases:
            ref = head.check(x, w, tok)
            want = ecc.ecc_linear_logprob_grad(x, w, tok, ref.lse, None, dlp)
            assert all(torch.equal(a, b) for a, b in zip(r[:3], ref[:3])) and all(torch.equal(a, b) for a, b in zip(g[:2], want[:2]))
            assert int(status.item()) == 0


def test_gated_calls_in_a_row_share_a_workspace():
    gen = torch.Generator("cuda").manual_seed(10)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    M, N, K = 300, 1500, 517                              # rows off 16-byte boundaries: copies in the workspace
    sets = [[gated.rows_of(gen, r, c, BF16) for r, c in ((M, K), (N, K), (N, K), (M, N), (M, N), (M, N))] for _ in range(3)]
    alone = []
    for x, wg, wu, dy, g, u in sets:
        alone.append((gated.check(x, wg, wu, scale=0.05), gated.check_grad(dy, x, wg, wu, g, u, scale=0.05)))
    got = [(ecc.ecc_gated_linear(x, wg, wu, scale=0.05, ws=ws)[0], ecc.ecc_gated_linear_grad(dy, x, wg, wu, g, u, scale=0.05, ws=ws))
           for _ in range(3) for x, wg, wu, dy, g, u in sets]
    torch.cuda.synchronize()
    for i, (y, r) in enumerate(got):
        assert torch.equal(y, alone[i % 3][0]) and all(torch.equal(a, b) for a, b in zip(r, alone[i % 3][1]))


def test_two_streams_at_once():
    """The same operators on two streams at the same time, small and large, with their own tensors."""
    gen = torch.Generator("cuda").manual_seed(11)
    jobs = []
    for M, N, V, K in ((40, 600, 3000, 192), (700, 3000, 20000, 640)):
        x, wg, wu, w = (gated.rows_of(gen, r, K, BF16, std=s) for r, s in ((M, 1.0), (N, 0.1), (N, 0.1), (V, 0.1)))
        dy, tok, dlp = gated.rows_of(gen, M, N, BF16), head.tokens_of(gen, M, V), torch.randn(M, generator=gen, device="cuda")

        def job(x=x, wg=wg, wu=wu, w=w, dy=dy, tok=tok, dlp=dlp, M=M, N=N, stream=None):
            g, u = (torch.empty(M, N, dtype=BF16, device="cuda") for _ in range(2))
            y, _ = ecc.ecc_gated_linear(x, wg, wu, pre_gate=g, pre_up=u, stream=stream)
            r = ecc.ecc_linear_logprob(x, w, tok, stream=stream)
            a = ecc.ecc_gated_linear_grad(dy, x, wg, wu, g, u, stream=stream)
            b = ecc.ecc_linear_logprob_grad(x, w, tok, r.lse, r.entropy, dlp, stream=stream)
            p = wg.float()
            state = ecc.adamw_state([p], 8)
            for step in (1, 2):
                ecc.ecc_adamw([p], [a[1]], state, step=step, stream=stream)
            return [y, *r, *a, *b, p, *state.m, *state.v]

        jobs.append((job, job()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(5):
        got = []
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        for (job, _), s in zip(jobs * 2, streams[::-1] + streams):
            with torch.cuda.stream(s):
                got.append(job())
        torch.cuda.synchronize()
        for (_, want), g in zip(jobs * 2, got):
            assert all(torch.equal(a, b) for a, b in zip(want, g))
