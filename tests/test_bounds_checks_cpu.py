"""The debug-bounds build checks the accesses of every kernel: each unit with a kernel that
takes operands names a check for every kind of buffer that it has.  (What the checks find is seen on
a GPU: tests/test_gpu_debug_bounds.py, tests/test_gpu_routing_block.py, tests/test_gpu_routing_bounds.py.)"""
import os
import re

import pytest

from block_scaled_fp8_w8a8_gb300 import build

# Inputs, a second input, outputs, scales or weights, workspace, shared memory: the sites.
A, B, C, S, W, M = ("SITE_BOUNDS_" + s for s in ("A", "B", "C", "SCALES", "WORKSPACE", "SMEM"))
NEEDS = {
    "route.cu": ({A, B, C, W, M}, ["group.cuh"]),
    "combine.cu": ({A, B, C, S}, []),
    "adapter.cu": ({A, B, C, S}, ["adapter.cuh"]),
    "adapter_tile.cu": ({A, B, C, S, W}, ["adapter.cuh"]),
}
NO_OPERANDS = {"api.cu", "status.cu", "hostio.cu", "noalloc.cu"}    # no kernel, or copies by whole pieces


def code(*names):
    text = "".join(open(os.path.join(build.SRC, n)).read() for n in names)
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


@pytest.mark.parametrize("unit", [u for u in build.UNITS if u not in NO_OPERANDS])
def test_every_unit_with_a_kernel_has_checks(unit):
    assert "__global__" in code(unit)
    sites, headers = NEEDS.get(unit, (set(), []))
    text = code(unit, *headers)
    assert "in_bounds(" in text
    missing = {s for s in sites if s not in text}
    assert not missing, missing


# Buffers of the calls, as the kernels read and write them by index: each line with such an access has a
# check on it, or stands below the line that has it.
INDEXED = {
    "route.cu": r"\bp\.(?:valid|bias|ids|weights)\[|p\.out\.(?:order|offsets|rows|rank|hist)\[",
    "group.cuh": r"\bg\.(?:order|offsets|rows|rank|hist)\[",
    "adapter.cuh": r"\bp\.(?:order|offsets|scales)\[",
    "adapter.cu": r"\bp\.(?:order|offsets|scales)\[",
    "adapter_tile.cu": r"\bp\.a\.(?:order|offsets|scales)\[",
}
CHECK = r"in_bounds\(|is_\w+(?:<\w+>)?\(|\.holds\("


@pytest.mark.parametrize("name", INDEXED)
def test_indexed_accesses_stand_by_a_check(name):
    lines = code(name).split("\n")
    for i, line in enumerate(lines):
        if re.search(INDEXED[name], line):
            assert re.search(CHECK, "\n".join(lines[max(0, i - 4):i + 1])), f"{name}: {line.strip()}"
