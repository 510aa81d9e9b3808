"""The build refuses a library whose statistics' kernels did not get the number
of registers that their warps share out (each call with many tokens would be
refused)."""
import pytest

from lossless_entropy_coding_gb300 import build

NAME = "_ZN3ecc16gemm_pair_kernelILb0ELb0ELb{}ELi{}EEEv14CUtensorMap_stS1_NS_8GemmArgsE"


def report(*kernels):
    return "ptxas info    : 0 bytes gmem\n" + "".join(
        f"ptxas info    : Compiling entry function '{name}' for 'sm_103a'\n"
        f"ptxas info    : Function properties for {name}\n    8 bytes stack frame, 12 bytes spill stores, 24 bytes spill loads\n"
        f"ptxas info    : Used {n} registers, used 1 barriers, 240 bytes smem\n" for name, n in kernels)


def test_the_number_of_registers():
    other = (NAME.format(0, 4), 106)
    build.check_registers(report(other, (NAME.format(0, 3), 168), (NAME.format(1, 3), 168)), build.STATS_KERNELS, 168)
    for kernels in ((other,), (other, (NAME.format(0, 3), 168)), ((NAME.format(0, 3), 168), other, (NAME.format(1, 3), 160)),
                    ((NAME.format(0, 3), 170), (NAME.format(1, 3), 170)), ()):
        with pytest.raises(RuntimeError, match="registers"):
            build.check_registers(report(*kernels), build.STATS_KERNELS, 168)
