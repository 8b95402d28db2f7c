"""CPU test of the sources: a kernel that lets itself be scheduled beside its
predecessor (griddep_release) has not waited for the grids before, so it reads
the call's inputs through the L2 and not through the read-only path."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sm_b200", "csrc")


def kernels():
    """(file, kernel name, body) of every __global__ function."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"__global__", text):
            at = text.index("{", m.end())
            name = re.findall(r"(\w+)\s*\(", text[m.end():at])
            depth, end = 0, at
            while True:
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                end += 1
                if depth == 0:
                    break
            yield os.path.basename(path), [n for n in name if n != "__launch_bounds__"][-1], text[at:end]


def test_every_kernel_waits():
    for path, name, body in kernels():
        assert "griddep_wait()" in body or "griddep_join()" in body or "merge_prologue(" in body, (path, name)


def test_early_kernels_read_through_the_l2():
    early = [(path, name, body) for path, name, body in kernels() if "griddep_release()" in body]
    assert {name for _, name, _ in early} == {"window_kernel", "paged_prepare_kernel"}
    for path, name, body in early:
        assert not re.search(r"__ldg\s*\(", body), (path, name)
