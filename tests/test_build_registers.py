"""The build's look at the registers that a kernel is launched with (CPU only)."""
import re

import pytest

from accept_select_top_gb300 import build as B

LOG = """ptxas info    : 0 bytes gmem
ptxas info    : Compiling entry function '_ZN4spec6kernelILi64EEEvNS_4ArgsE' for 'sm_103a'
ptxas info    : Function properties for _ZN4spec6kernelILi64EEEvNS_4ArgsE
    8 bytes stack frame, 92 bytes spill stores, 88 bytes spill loads
ptxas info    : Used 80 registers, used 1 barriers, 8 bytes cumulative stack size
ptxas info    : Compiling entry function '_ZN4spec5otherILi64EEEvNS_4ArgsE' for 'sm_103a'
ptxas info    : Used 53 registers, used 0 barriers
ptxas info    : Compiling entry function '_ZN4spec6kernelILi128EEEvNS_4ArgsE' for 'sm_103a'
ptxas info    : Used {} registers, used 1 barriers
"""


def test_every_instance_counts():
    B.check_registers(LOG.format(80), "kernel", 80)
    for log, kernel in ((LOG.format(72), "kernel"), (LOG.format(80), "missing"), ("", "kernel")):
        with pytest.raises(RuntimeError, match="80 registers"):
            B.check_registers(log, kernel, 80)


def test_the_checked_kernels_are_there():
    """Each entry names a source, a kernel in it and the number that the source is written for."""
    import os
    for name, (kernel, want) in B.REGISTERS.items():
        text = open(os.path.join(B.CSRC, name)).read()
        assert kernel in text and int(re.search(r"kRegs = (\d+)", text).group(1)) == want


def test_every_register_split_is_checked():
    for src in B.sources():
        if "setmaxnreg" in open(src).read():
            assert src.rsplit("/", 1)[-1] in B.REGISTERS
