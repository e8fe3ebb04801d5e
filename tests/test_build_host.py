"""The build's own checks (no GPU)."""
import os

import pytest

from online_softmax_attention_zigzag_gb300 import build

SRC = "static constexpr int kStartRegs = E4M3 ? 96 : 128, kOther = 1;"


def _log(regs):
    """What ptxas prints for the eight kernels; regs: of the e4m3 ones and of the bf16 ones."""
    out = "ptxas info    : 0 bytes gmem\n"
    for d in (64, 128):
        for e4m3 in (0, 1):
            for alone in (0, 1):
                out += (f"ptxas info    : Compiling entry function '_ZN2ra18paged_chunk_kernelILi{d}ELb{e4m3}ELb{alone}EEEvNS_1PE' for 'sm_103a'\n"
                        "ptxas info    : Function properties for x\n    8 bytes stack frame, 0 bytes spill stores\n"
                        f"ptxas info    : Used {regs[1 - e4m3]} registers, used 3 barriers\n")
    return out


def test_registers_that_the_split_counts_on():
    build.check_registers("a.cu", SRC, _log((96, 128)))
    build.check_registers("b.cu", "no such kernel", "")


@pytest.mark.parametrize("regs,match", [((104, 128), "e4m3.*104 registers.*96"), ((96, 120), "bf16.*120 registers.*128")])
def test_other_registers_are_refused_with_a_reason(regs, match):
    with pytest.raises(RuntimeError, match=match):
        build.check_registers("a.cu", SRC, _log(regs))


def test_kernels_that_are_not_in_the_log():
    with pytest.raises(RuntimeError, match="8 expected"):
        build.check_registers("a.cu", SRC, "")


def test_the_source_states_them():
    """The check reads the constant that the kernel's split is built on."""
    with open(os.path.join(build.CSRC, "paged_chunk.cu")) as f:
        text = f.read()
    with pytest.raises(RuntimeError, match="8 expected"):
        build.check_registers("paged_chunk.cu", text, "")
    build.check_registers("paged_chunk.cu", text, _log((96, 128)))
