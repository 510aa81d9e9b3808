"""Scratch sizes of jobs that the calls refuse: a caller asks for them before
the call checks anything, so no job may stop the process there (run in a
process of its own, which a trap would end)."""
import subprocess
import sys

from test_lm_more_arguments import P
import lossless_entropy_coding_gb300 as ecc

CODE = """
import sys
sys.path[:0] = {path!r}
import test_lm_more_arguments as t
import lossless_entropy_coding_gb300 as ecc
F = (t.math.nan, t.math.inf, 1.0)
f = ecc.lib().ecc_linear_logprob_workspace_bytes
for rows, vocab, K in ((4, 0, 16), (0, 0, 0), (0, 0, 16), (1 << 31, 0, 16), (4, 1 << 31, 16), ((1 << 64) - 1, 1, 1), (4, 8, 1 << 31)):
    for scale in F:
        assert f(t.HEAD.pack(t.P, t.P, 0, 0, 0, 0, rows, vocab, K, K, K, scale, ecc.BF16, 0)) == 0 or (rows < 1 << 31 and vocab and scale == 1)
f = ecc.lib().ecc_linear_logprob_grad_workspace_bytes
for rows, vocab, K in ((4, 0, 16), (0, 0, 0), (0, 0, 16), (1 << 31, 0, 16), (1 << 31, 8, 16), (4, 1 << 31, 16), ((1 << 64) - 1, 1, 1), (4, 8, 1 << 31)):
    for dx in (0, t.P):
        for scale in F:
            assert f(t.HEAD_GRAD.pack(t.P, t.P, 0, t.P, 0, 0, 0, dx, t.P, rows, vocab, K, K, K, K, K, scale, ecc.BF16, ecc.BF16, 0)) == 0
for name, s in (("ecc_gated_linear", t.GATED), ("ecc_gated_linear_grad", t.GATED_GRAD)):
    f = getattr(ecc.lib(), name + "_workspace_bytes")
    for value in (0, 1, (1 << 31) - 1, (1 << 64) - 1):
        kinds = [{{"P": min(value, 1 << 20), "Q": value, "f": 1.0, "I": value & 15}}[c] for c in expand(s.format)]
        f(s.pack(*kinds))
print("done")
"""
EXPAND = """
import re
def expand(fmt):
    return "".join(c * int(n or 1) for n, c in re.findall(r"(\\d*)([PQfId])", fmt))
"""


def test_scratch_sizes_of_refused_jobs():
    r = subprocess.run([sys.executable, "-c", EXPAND + CODE.format(path=sys.path)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "done" in r.stdout, (r.returncode, r.stderr)


def test_a_head_without_a_vocabulary_is_refused():
    from test_lm_more_arguments import head, head_grad
    for kw in (dict(vocab=0), dict(vocab=0, rows=0), dict(vocab=0, K=0)):
        assert head(ws=P, ws_bytes=1 << 30, **kw) == head_grad(ws=P, ws_bytes=1 << 30, **kw) == ecc.ERR_ARG


def test_scales_whose_product_with_log2_e_is_infinite():
    from test_lm_more_arguments import head, head_grad
    for scale in (2.0**127, -(2.0**127), 3e38):
        assert head(ws=P, ws_bytes=1 << 30, scale=scale) == head_grad(ws=P, ws_bytes=1 << 30, scale=scale) == ecc.ERR_ARG
