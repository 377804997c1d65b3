"""The many-rows chains of the 8-bit experts at their edges, against the float64 oracle (bounds:
test_fp8_gpu.py)."""
import numpy as np
import pytest
import torch

import combine_router_softmax_top_gb300 as moe
import test_fp8_gpu as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from combine_router_softmax_top_gb300 import build
    build.build()
    torch.cuda.init()


def kernels(run):
    """Names of the kernels that run() launches."""
    moe.moe_profile_start(64)
    run()
    torch.cuda.synchronize()
    return [n for n, _ in moe.moe_profile_stop()]


def test_a_pair_claims_more_tiles_than_its_mailbox_has_slots():
    # 480000 rows: 1900 row tiles of each product, some 50 a CTA pair, three times
    # round the 16 slots; one column tile, so that tiles are as short as they can be
    c = G.Case(T=60000, H=64, E=8, k=8, F=64, kind="balanced", seed=41)
    c.quantize()
    c.permute()
    for _ in range(3):
        for t in (c.o, c.dx):
            t.fill_(7.0)
        assert "fp8_gemm_ffn_fwd" in kernels(c.forward)
        c.combine_bwd()
        c.dgrad()
        c.status()
        G.test_forward_stages(c)
        G.test_dgrad_stages(c)
