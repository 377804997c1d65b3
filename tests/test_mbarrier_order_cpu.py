"""An mbarrier is used by a block's threads only behind its initialisation: read from the kernels'
source (CPU), since a run shows the opposite only when one warp happens to be late."""
import os
import re

import pytest

from test_fp4_source_cpu import body, code

# What touches an mbarrier, in this CTA or (through an address of the cluster) in another one.
USES = r"\b(?:mbar_\w+|umma_commit\w*|tma_load\w*|bulk_load|arrive_remote|arrive)\("
REMOTE = r"\b(?:mapa_shared|umma_commit_pair|tma_load_2d_pair)\("
KERNELS = ["rows_fp4.cu", "grouped_gemm_fp4.cu", "rows_fp8.cu", "grouped_gemm_fp8.cu",
           "grouped_gemm.cu"]


def helpers(text):
    """name -> body of the file's device functions."""
    found = {}
    for m in re.finditer(r"__device__ __forceinline__ [\w<>&* ]+?(\w+)\(", text):
        found[m[1]] = found.get(m[1], "") + body(text, m.end())
    return found


def using(fns, pattern):
    """Names of the functions that match the pattern themselves or through others."""
    names = {n for n, b in fns.items() if re.search(pattern, b)}
    while True:
        call = r"\b(?:%s)(?:<[^;()]*>)?\(" % "|".join(sorted(names) or ["$^"])
        more = {n for n, b in fns.items() if n not in names and re.search(call, b)}
        if not more:
            return names
        names |= more


def at_top(text, pattern):
    """Places of the pattern that no condition or loop encloses."""
    depth, out = 0, []
    places = {m.start() for m in re.finditer(pattern, text)}
    for i, ch in enumerate(text):
        if i in places and depth == 1:  # (text starts with the kernel's own brace)
            out.append(i)
        depth += (ch == "{") - (ch == "}")
    return out


def first_uses(text):
    """Of every kernel that initialises mbarriers: (its end of the initialisation, block barriers
    and cluster barriers behind that, first use in this CTA, first use in the cluster)."""
    fns = helpers(text)
    local, remote = using(fns, USES), using(fns, REMOTE)
    for m in re.finditer(r"__global__ ", text):
        b = body(text, m.end())
        inits = [i.end() for i in re.finditer(r"\bmbar_init\(|fence_mbar_init\(", b)]
        if not inits:
            continue
        end = max(inits)

        def first(names, pattern):
            call = r"\b(?:%s)(?:<[^;()]*>)?\(" % "|".join(sorted(names) or ["$^"])
            at = [u.start() for p in (call, pattern) for u in re.finditer(p, b) if u.start() > end]
            assert at, "nothing uses the barriers"
            return min(at)

        yield (end, [i for i in at_top(b, r"__syncthreads\(\)") if i > end],
               [i.start() for i in re.finditer(r"cluster_sync\(\)", b) if i.start() > end],
               first(local, USES), first(remote, REMOTE) if remote else None)


@pytest.mark.parametrize("name", KERNELS)
def test_no_use_of_an_mbarrier_before_its_initialisation_is_everyones(name):
    found = list(first_uses(code(name)))
    assert found
    for end, blocks, clusters, local, remote in found:
        assert blocks and blocks[0] < local, "no barrier of the block between the two"
        if remote is not None:
            assert clusters and clusters[0] < remote, "no barrier of the cluster between the two"


def test_the_rule_sees_an_early_arrival():
    text = ("__device__ __forceinline__ void post(C& c) { ptx::mbar_arrive(&c.full); }\n"
            "__global__ void k() { if (t == 0) { ptx::mbar_init(&c.full, 1); ptx::fence_mbar_init(); }"
            " %s if (t == 64) { %s post(c); } __syncthreads(); }")
    for top, inner, fine in (("__syncthreads();", "", True), ("", "", False),
                             ("", "__syncthreads();", False)):
        (end, blocks, _, local, _), = first_uses(text % (top, inner))
        assert (blocks[0] < local) == fine
