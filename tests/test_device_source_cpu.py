"""Rules of the device code that no run on one GPU can show broken, read from its source."""
import glob
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCES = sorted(glob.glob(os.path.join(ROOT, "combine_router_softmax_top_gb300", "csrc", "*.cu*")))


def code(path):
    """The source without comments, adjacent string literals joined."""
    s = open(path).read()
    s = re.sub(r"//[^\n]*", "", s)
    s = re.sub(r"/\*.*?\*/", "", s, flags=re.S)
    return re.sub(r'"\s*\n?\s*"', "", s)


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_load_is_multicast(path):
    """The library runs with one rank on each of several GPUs: a TMA load fills its own CTA's
    shared memory alone. (tcgen05.commit may arrive on the barriers of a CTA pair.)"""
    for s in re.findall(r'"(?:[^"\\]|\\.)*"', code(path)):
        for instruction in s.replace("\\n", ";").replace("\\t", " ").split(";"):
            assert not ("cp.async.bulk" in instruction and "multicast" in instruction), instruction
