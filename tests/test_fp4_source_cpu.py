"""Rules of the 4-bit kernels' device code that no run on one GPU can show broken, read from its
source (CPU)."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "combine_router_softmax_top_gb300", "csrc")


def code(name):
    s = open(os.path.join(CSRC, name)).read()
    s = re.sub(r"//[^\n]*", "", s)
    return re.sub(r"/\*.*?\*/", "", s, flags=re.S)


def body(text, start):
    """From the first brace after `start` to the one that closes it."""
    at = text.index("{", start)
    depth = 0
    for i in range(at, len(text)):
        depth += (text[i] == "{") - (text[i] == "}")
        if depth == 0:
            return text[at:i]
    raise AssertionError("no end")


def arguments(text, at):
    """Of the call whose parenthesis opens before `at`."""
    depth, i = 1, at
    while depth:
        depth += (text[i] == "(") - (text[i] == ")")
        i += 1
    return text[at:i - 1]


def functions(name, names):
    text = code(name)
    return {m[1]: body(text, m.end()) for m in re.finditer(r"\bint (%s)\(" % "|".join(names), text)}


def test_a_claimed_tiles_slot_is_released_by_its_readers():
    """The slot that a claimed tile is read from is overwritten once its readers have arrived: a
    relaxed arrival would not order their reads before that, nor one at the scope of a CTA where the
    writer is in another one."""
    local, remote = "mbar_arrive", "mbar_arrive_cluster"
    seen = []
    for name, names in (("grouped_gemm_fp4.cu", ("mailed_tile", "handed_tile")),
                        ("rows_fp4.cu", ("claimed_tile",))):
        for fn, text in functions(name, names).items():
            for call, args in re.findall(r"(\w*arrive\w*)\(([^;]*);", text):
                seen.append((fn, call, re.search(r"c\.(\w+)", args)[1]))
    assert seen == [("mailed_tile", remote, "mail_empty"), ("mailed_tile", local, "hand_full"),
                    ("handed_tile", local, "hand_empty"), ("claimed_tile", local, "claim_empty")]


def test_every_wait_has_a_limit():
    """No loop waits for memory that another thread writes without looking at the time."""
    for name in ("grouped_gemm_fp4.cu", "rows_fp4.cu"):
        text = code(name)
        assert "mbar_try_wait(" not in text  # (the unbounded primitive)
        for m in re.finditer(r"while \(ld_acquire\(", text):
            assert "kWaitLimitNs" in body(text, m.end())
        waits = [arguments(text, m.end()) for m in re.finditer(r"\bmbar_wait\(", text)]
        assert waits and all("kWaitLimitNs" in w for w in waits), waits


def test_a_copy_of_scales_starts_on_an_even_row():
    """A bulk copy starts on a 16-byte boundary: two rows of 8 scale bytes."""
    for name in ("grouped_gemm_fp4.cu", "rows_fp4.cu"):
        text = code(name)
        assert re.search(r"t\.row & ~1ll|row & ~1ll", text) and "scale_rows(p.N)" in text
    assert "(n + 1) & ~1ll" in code("fp4_mma.cuh")
