"""What `python -m lossless_entropy_coding_gb300.build` builds: the library
needs no PyTorch; the module that unpacks its tensors is built where PyTorch
is there, next to the library it is linked with (not for the checked one)."""
import subprocess
import sys

import pytest

from conftest import ROOT

PROGRAM = """
import sys
if {without_torch}:
    sys.modules["torch"] = None          # import torch raises ImportError
import lossless_entropy_coding_gb300.build as b
built = []
b.build = lambda force=False, checked=False: built.append("checked" if checked else "library") or "lib"
compile_torch = b.build_torch
def build_torch(force=False):
    if {without_torch}:
        return compile_torch(force)      # as it is: it needs PyTorch's headers
    built.append("torch")
    return "module"
b.build_torch = build_torch
b.main({args})
print(built)
"""


@pytest.mark.parametrize("args,without_torch,want", [([], True, ["library"]), (["--checked"], True, ["checked"]),
                                                     (["--checked"], False, ["checked"]), ([], False, ["library", "torch"])])
def test_build_command(args, without_torch, want):
    r = subprocess.run([sys.executable, "-c", PROGRAM.format(args=args, without_torch=without_torch)], cwd=ROOT,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert r.stdout.splitlines()[-1] == str(want)
    assert ("PyTorch" in r.stderr) == (without_torch and not args)
