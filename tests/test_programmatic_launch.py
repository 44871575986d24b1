"""Kernels that are launched before their stream's last kernel has ended take no read-only loads.

Such a kernel is resident while the kernel before it still writes what it is about to read.  Read-only loads
(ld.global.nc, __ldg) are defined only for data that nothing writes in the kernel's lifetime, however late in it they are
issued; ordinary loads see the writes once the wait is over.  No run shows the difference, so the sources are read."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "stencil_conv2d_fwd_gb300", "csrc")


def code(path):
    with open(path) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


WAITING = sorted(os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "*.cu")) if re.search(r"\bpdl_wait\(\)", code(p)))


def test_the_files_are_found():
    assert {"linear_rows.cu", "linear_tc.cu", "kv_quantize.cu", "residual_norm.cu", "attn_q8.cu", "attn_tc.cu", "attn_join.cu"} <= set(WAITING)


@pytest.mark.parametrize("name", WAITING)
def test_no_read_only_load_beside_a_wait(name):
    text = code(os.path.join(CSRC, name))
    readers = {"__ldg", r"ld\.global\.nc"}
    for header in glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")):
        # functions of the shared headers whose body is such a load
        readers |= {m.group(1) for m in re.finditer(r"(\w+)\([^()]*\)\s*\{[^{}]*ld\.global\.nc", code(header))}
    assert "ldg16" in readers
    for r in readers:
        assert not re.search(rf"(?<![\w.]){r}\b", text), f"{name}: {r}"
