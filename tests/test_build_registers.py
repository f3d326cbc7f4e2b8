"""The build refuses kernels whose register count is not the one their setmaxnreg
split counts on."""
import os
import re

import pytest

from paged_kv_attention_36_b200 import build

LOG = """ptxas info    : Compiling entry function '_ZN2pa17prefill_i8_kernelILi64ELi4ELb0EEEv' for 'sm_100a'
ptxas info    : Function properties for _ZN2pa17prefill_i8_kernelILi64ELi4ELb0EEEv
    8 bytes stack frame, 4 bytes spill stores, 4 bytes spill loads
ptxas info    : Used {n} registers, used 3 barriers, 8 bytes cumulative stack size
ptxas info    : Compiling entry function '_ZN2pa13append_kernelENS_12AppendParamsE' for 'sm_100a'
ptxas info    : Function properties for _ZN2pa13append_kernelENS_12AppendParamsE
    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used 26 registers, used 0 barriers
"""


def test_check_registers():
    assert build.check_registers(LOG.format(n=80)) == 1
    assert build.check_registers("") == 0
    for n in (72, 79, 88):
        with pytest.raises(RuntimeError, match="80"):
            build.check_registers(LOG.format(n=n))


def test_the_number_is_the_kernels():
    source = open(os.path.join(build.CSRC, "pa_prefill_i8.cuh")).read()
    regs, soft, convert, issue = (int(re.search(rf"\b{name} = (\d+)", source).group(1)) for name in
                                  ("kRegs", "kSoftmaxRegs", "kConvertRegs", "kIssueRegs"))
    assert build.REGISTERS["prefill_i8_kernel"] == regs and soft + convert + issue <= 3 * regs
