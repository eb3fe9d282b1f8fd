"""include/moe.h in programs of its callers: fp16 scales are read and written through their own type, as C and as C++."""
import os
import subprocess

import pytest

INCLUDE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")

CALLER = """
#include "moe.h"
const uint16_t *int8_scales(const moe_weights *w) { const uint16_t *s = w->gate.scale; return s + 1; }
unsigned first_scale(const moe_weights *w) { return w->down.scale[0]; }
moe_mat int8_mat(const int8_t *q, const uint16_t *scale) { moe_mat m = {q, scale}; return m; }
void set_scale(moe_mat *m, const uint16_t *scale) { m->scale = scale; }
"""
E4M3 = """
moe_mat e4m3_mat(const uint8_t *q, const float *scale) { moe_mat m = {q, (const uint16_t *)scale}; return m; }
"""


@pytest.mark.parametrize("cc", [("gcc", "-x", "c", "-std=c11"), ("g++", "-x", "c++", "-std=c++11")], ids=["c", "c++"])
@pytest.mark.parametrize("source", [CALLER, CALLER + E4M3], ids=["int8", "e4m3"])
def test_callers_compile(cc, source):
    r = subprocess.run([*cc, "-Wall", "-Wextra", "-Werror", "-fsyntax-only", "-I", INCLUDE, "-"], input=source,
                       text=True, capture_output=True)
    assert r.returncode == 0, r.stderr
