"""No kernel that may start while the one before it is at work loads through the
read-only path: it wants memory that nothing writes while the kernel runs.  A
wrong value would show only now and then, so the sources are read instead."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "combine_routing_count_prefix_gb300", "csrc")
# launched cooperatively, after everything before it
EXCEPTED = ("dispatch_signaled_kernel",)


def code(path):
    """The source without comments and without the excepted kernels' bodies."""
    with open(path) as f:
        s = re.sub(r"//[^\n]*", "", f.read())
    for name in EXCEPTED:
        at = s.find(f"{name}(Geometry")
        if at >= 0:
            s = s[:at] + s[s.index("\n}\n", at):]
    return s


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.cu*"))), ids=os.path.basename)
def test_no_read_only_loads(path):
    found = re.findall(r"__ldg\s*\(|ld\.global\S*\.nc", code(path))
    assert not found, found
