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


def rest_of_block(text):
    """Up to the brace that closes the block in which the text begins."""
    depth = 0
    for i, c in enumerate(text):
        depth += (c == "{") - (c == "}")
        if depth < 0:
            return text[:i]
    return text


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_load_is_multicast(path):
    """The library runs with one rank on each of several GPUs: a TMA load fills its own CTA's
    shared memory alone. (tcgen05.commit may arrive on the barriers of a CTA pair.)"""
    for s in re.findall(r'"(?:[^"\\]|\\.)*"', code(path)):
        for instruction in s.replace("\\n", ";").replace("\\t", " ").split(";"):
            assert not ("cp.async.bulk" in instruction and "multicast" in instruction), instruction


def test_an_announced_stage_is_loaded_whole():
    """A producer that gives up leaves no stage of its operand ring with some of the announced
    bytes on their way: after an abort the loads in flight are waited for by whole stages
    (drain_loads), so none may write into shared memory that is no longer the kernel's."""
    seen = 0
    for path in SOURCES:
        text = code(path)
        if "drain_loads(" not in text:
            continue
        for at in re.finditer(r"mbar_arrive_expect_tx\(", text):
            stage = rest_of_block(text[at.start():])
            if "tma_load" in stage:
                seen += 1
                assert "return" not in stage, (os.path.basename(path), stage)
    assert seen >= 2


def test_a_claimed_tiles_slot_is_released_by_its_readers():
    """The slot that a claimed tile is read from is overwritten once its readers have arrived: a
    relaxed arrival would not order their loads before that, nor one at the scope of a CTA
    where the writer is in another one."""
    seen = []
    for path in SOURCES:
        text = code(path)
        for at in re.finditer(r"int (next_tile|take_tile)\([^;{]*\{", text):
            for a in re.findall(r"(\w*arrive\w*)\(([^;]*);", rest_of_block(text[at.end():])):
                seen.append((os.path.basename(path), at[1], a[0], re.search(r"c\.(\w+)", a[1])[1]))
    local, remote = "mbar_arrive", "mbar_arrive_cluster"
    assert seen == [("grouped_gemm_fp8.cu", "take_tile", remote, "mail_empty"),
                    ("grouped_gemm_fp8.cu", "take_tile", local, "sched_full"),
                    ("grouped_gemm_fp8.cu", "next_tile", local, "sched_empty"),
                    ("rows_fp8.cu", "next_tile", local, "sched_empty")]
    ptx = code(os.path.join(ROOT, "combine_router_softmax_top_gb300", "csrc", "sm100_ptx.cuh"))
    assert "mbarrier.arrive.release.cluster.shared::cluster.b64" in ptx
    assert "mbarrier.arrive.relaxed" not in ptx
