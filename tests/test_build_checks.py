"""What the build checks of the compiler's output (no GPU)."""
import os
import subprocess

import pytest

from serial_draft_head_gb300 import _build

NAME = "_ZN6dspark4tree47_GLOBAL__N__24f4ff91_14_tree_attend_cu_6a12698213attend_kernel%sEvNS0_10AttendArgsE"
LOG = """ptxas info    : 0 bytes gmem
ptxas info    : Compiling entry function '%s' for 'sm_103a'
ptxas info    : Function properties for %s
    72 bytes stack frame, 192 bytes spill stores, 196 bytes spill loads
ptxas info    : Used %d registers, used 2 barriers, 72 bytes cumulative stack size
"""


def log(args, used):
    return LOG % (NAME % args, NAME % args, used)


def test_a_kernel_with_other_registers_than_it_counts_on_fails_the_build():
    good = log("ILb0ELb1ELi128ELi96EE", 96) + log("ILb1ELb0ELi64ELi128EE", 128)
    assert _build.check_registers(good) == 2
    for used in (95, 80, 128):
        with pytest.raises(RuntimeError, match="counts on 96"):
            _build.check_registers(good + log("ILb1ELb1ELi64ELi96EE", used))
    # other kernels may have any number
    other = LOG.replace("%s", "_ZN6dspark4tree11join_kernelILb0ELi128EEEvNS0_10AttendArgsE") % 40
    assert _build.check_registers(other) == 0


def test_the_kernels_of_this_tree_are_found(tmp_path):
    """The report of tree_attend.cu as it stands: all eight kernels, each with its number; and no
    other check of it is left to the making of a handle."""
    src = os.path.join(_build.CSRC, "tree_attend.cu")
    res = subprocess.run([_build.nvcc()] + _build.ARCH + [
        "-O3", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr", "-Xptxas", "-v",
        "-I", os.path.join(_build.ROOT, "include"), "-c", src, "-o", str(tmp_path / "x.o")],
        capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    assert _build.check_registers(res.stderr) == 8
    assert "numRegs" not in open(src).read()
