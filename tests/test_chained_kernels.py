"""Kernels that may start while an earlier kernel of their call still runs must not read what
that one writes as constant data: neither by __ldg and its like nor through a const __restrict__
pointer, which the compiler may read before the kernel's wait.  Read off the sources."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "chunked_gated_delta_fwd_gb300", "csrc")
# what one kernel of a call hands to another, by file
HANDED_ON = {
    "kda_linear_simt.cu": {"chunk_off", "tab", "local", "gam", "states"},
    "kda_linear_tc.cu": {"first", "tab", "n_segs", "order", "ticket", "s_end", "s_in", "decay",
                         "seg_decay"},
}


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_every_file_with_chained_launches_is_read():
    found = {n for n in os.listdir(CSRC) if n.endswith(".cu") and "launch_chained(" in source(n)}
    assert found == set(HANDED_ON)


@pytest.mark.parametrize("name", sorted(HANDED_ON))
def test_no_constant_loads_of_what_a_call_hands_on(name):
    s = source(name)
    for arg in re.findall(r"\b__ld(?:g|cs|cg|ca|lu|cv)\(([^;]*);", s):
        assert not HANDED_ON[name] & set(re.findall(r"\w+", arg)), arg
    for kernel in re.findall(r"__global__[^;{]*\{", s):
        for const, param in re.findall(r"(const\s+)?[\w]+\*\s*__restrict__\s+(\w+)", kernel):
            assert not (const and param in HANDED_ON[name]), kernel


def test_a_state_updated_in_place_is_not_declared_apart():
    """hT may be h0: the kernel that takes both says nothing of them."""
    kernel = re.search(r"lin_scan_kernel\(([^)]*)\)", source("kda_linear_simt.cu")).group(1)
    assert "h0" in kernel and "hT" in kernel and "__restrict__" not in kernel
