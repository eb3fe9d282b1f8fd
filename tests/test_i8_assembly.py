"""i8_tile.hip's inline assembly sets M0 for each of its copies.  The compiler reserves M0, so a clobber of it cannot be
declared (hipcc warns and promises nothing): the kernels are right only while nothing that the compiler makes of them
uses M0 too, which this holds the build to."""
import os
import re
import subprocess
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from sparse_moe_layer_02_amd import build  # noqa: E402


def m0_lines(assembly):
    """(lines that use M0 within inline assembly, lines that use it elsewhere)."""
    within, elsewhere, inline = [], [], False
    for line in assembly.splitlines():
        if "#ASMSTART" in line:
            inline = True
        elif "#ASMEND" in line:
            inline = False
        elif re.search(r"\bm0\b", line.split(";")[0]):
            (within if inline else elsewhere).append(line.strip())
    return within, elsewhere


def test_a_use_by_the_compiler_is_seen():
    text = ";;#ASMSTART\n\ts_mov_b32 m0, s4\n;;#ASMEND\n\ts_mov_b32 m0, s5 ; m0\n\tv_mov_b32 v0, 1 ; m0\n"
    assert m0_lines(text) == (["s_mov_b32 m0, s4"], ["s_mov_b32 m0, s5 ; m0"])


def test_m0_is_the_inline_assemblys():
    r = subprocess.run([build.HIPCC, *build.FLAGS, "--offload-device-only", "-S", os.path.join(build.CSRC, "i8_tile.hip"),
                        "-o", "-"], text=True, capture_output=True)
    assert r.returncode == 0, r.stderr
    within, elsewhere = m0_lines(r.stdout)
    assert within and not elsewhere, elsewhere[:5]
