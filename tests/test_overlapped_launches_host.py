"""Kernels that begin under the previous launch of their stream (no GPU, from the sources)."""
import os
import re

from tests.conftest import ROOT

CSRC = os.path.join(ROOT, "routing_shared_expert_gb300", "csrc")


def text(name):
    with open(os.path.join(CSRC, name)) as fh:
        return re.sub(r"//[^\n]*", "", fh.read())


def with_includes(name, seen):
    seen.add(name)
    for inc in re.findall(r'#include "([^"]+)"', text(name)):
        if inc not in seen and os.path.exists(os.path.join(CSRC, inc)):
            with_includes(inc, seen)
    return seen


def test_no_read_only_loads_where_the_previous_launch_may_still_write():
    """A read-only load is defined only for data that nothing writes during the kernel's life, and
    these kernels are alive while the previous one writes: its output is often their operand."""
    overlapped = [f for f in sorted(os.listdir(CSRC)) if f.endswith(".cu") and "wait_for_previous()" in text(f)]
    assert len(overlapped) >= 5
    for f in overlapped:
        for part in with_includes(f, set()):
            found = re.findall(r"__ldg\s*\(|ld\.global\.nc|__restrict__", text(part))
            assert not found, f"{part} (in {f}): {found}"
