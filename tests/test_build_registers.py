"""The build looks whether the compiler gave the tile kernels the registers that their shares are made
for (no GPU and no compiler needed)."""
import importlib.util
import os

import pytest

PACKAGE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                       "draft_tree_construction_markov_b200")
spec = importlib.util.spec_from_file_location("_build_script", os.path.join(PACKAGE, "build.py"))
script = importlib.util.module_from_spec(spec)
spec.loader.exec_module(script)


def _log(*kernels):
    out = ["ptxas info    : 0 bytes gmem"]
    for name, regs in kernels:
        out += [f"ptxas info    : Compiling entry function '_ZN2dt12_GLOBAL__N_1{name}EEvNS0_6TcMapsE' for 'sm_100a'",
                f"ptxas info    : Function properties for _ZN2dt{name}",
                "    8 bytes stack frame, 4 bytes spill stores, 24 bytes spill loads",
                f"ptxas info    : Used {regs} registers, used 7 barriers, 8 bytes cumulative stack size"]
    return "\n".join(out)


GOOD = [("15paged_tc_kernelILi128ELi3ELi1", 80), ("15paged_tc_kernelILi64ELi2ELi2", 128),
        ("15paged_tc_kernelILi128ELi1ELi2", 168), ("15paged_tc_kernelILi64ELi1ELi1", 108), ("12other_kernel", 77)]


def test_the_numbers_that_the_shares_are_made_for_pass():
    script.check_registers(_log(*GOOD))
    script.check_registers(_log(("15paged_tc_kernelILi64ELi1ELi1", 96)))  # deals nothing out
    script.check_registers("")


@pytest.mark.parametrize("at,regs", [(0, 72), (1, 126), (2, 166)])
def test_another_number_is_an_error_of_the_build(at, regs):
    bad = list(GOOD)
    bad[at] = bad[at][0], regs
    with pytest.raises(RuntimeError, match=f"has {regs} registers"):
        script.check_registers(_log(*bad))


def test_the_table_says_what_the_source_says():
    src = open(os.path.join(PACKAGE, "csrc", "paged_tc.cu")).read()
    assert "kLaunchRegs = NQ == 1 ? 80 : kTma ? 168 : 128;" in src
    assert script.LAUNCH_REGS == {(1, 2): 168, (2, 1): 80, (3, 1): 80, (2, 2): 128, (3, 2): 128}
