"""The build refuses a kernel whose register split asks for more than it is launched with."""

import os
import re

import pytest

from paged_kv_cache_driven_b200 import build

UNIT = os.path.join(build.CSRC, "pa_k_rows.cu")
LOG = """ptxas info    : Compiling entry function '_ZN2pa11rows_kernelI6__halfLi128ELb1EEEv' for 'sm_100a'
ptxas info    : Function properties for _ZN2pa11rows_kernelI6__halfLi128ELb1EEEv
    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used 72 registers, used 3 barriers
ptxas info    : Compiling entry function '_ZN2pa11rows_kernelI6__halfLi64ELb1EEEv' for 'sm_100a'
ptxas info    : Used {} registers, used 3 barriers, 16 bytes cumulative stack size
"""


def test_too_few_registers_fail_the_build():
    for n in (80, 96):
        build.check_registers(UNIT, LOG.format(n))
    with pytest.raises(RuntimeError, match="72 registers"):
        build.check_registers(UNIT, LOG.format(72))
    with pytest.raises(RuntimeError, match="no register count"):  # the rule no longer finds it
        build.check_registers(UNIT, LOG.format(80).replace("Li64E", "Li65E"))
    build.check_registers(os.path.join(build.CSRC, "pa_k_rope.cu"), "")


def test_the_rule_is_the_kernels():
    text = open(os.path.join(build.CSRC, "pa_rows.cuh")).read()
    assert int(re.search(r"LAUNCH_REGS = (\d+)", text).group(1)) == \
        build.MIN_REGISTERS["pa_k_rows.cu"][1]
    assert "PASS_REGS = D == 64" in text
    assert "-v" in build.compile_command(UNIT)
