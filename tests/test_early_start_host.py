"""Rules of the kernels that may start while the kernel before them in the stream still
runs (sm100.cuh, launch_after), read from their sources: what that kernel writes is not
read-only for them, so nothing goes through the non-coherent path, and every such kernel
waits."""
import glob
import os
import re

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "chunk_routed_sparse_b200", "csrc")


def _code(path):
    with open(path) as f:
        text = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def _early():
    out = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        if re.search(r"launch_after\s*\(|ProgrammaticStreamSerialization", _code(path)):
            out.append(os.path.basename(path))
    return out


def _kernels(code):
    """(name, parameters, body) of every __global__ function."""
    for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\([^)]*\)\s*)?(\w+)\s*\(", code):
        at, depth = m.end(), 1
        while depth:
            depth += {"(": 1, ")": -1}.get(code[at], 0)
            at += 1
        params = code[m.end():at - 1]
        start = at = code.index("{", at) + 1
        depth = 1
        while depth:
            depth += {"{": 1, "}": -1}.get(code[at], 0)
            at += 1
        yield m.group(1), params, code[start:at]


def test_the_early_starting_files_are_found():
    assert {"k_rope.cu", "k_window_bwd.cu", "k_window_few.cu", "k_window_fwd.cu", "k_window_tile.cu"} <= set(_early())


@pytest.mark.parametrize("name", _early())
def test_early_starting_kernels_read_nothing_through_the_non_coherent_path(name):
    code = _code(os.path.join(CSRC, name))
    for bad in (r"ldg_nc16", r"ld\.global(\.\w+)*\.nc\b", r"\b__ldg\b", r"\b__ldlu\b"):
        assert not re.search(bad, code), bad
    found = list(_kernels(code))
    assert found
    for kernel, params, body in found:
        assert not re.search(r"const\s+\w+\s*\*\s*__restrict__", params), kernel
        assert "wait_for_previous_kernel()" in body, kernel
