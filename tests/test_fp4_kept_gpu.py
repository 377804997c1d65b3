"""The 4-bit expert products: h's scale bytes beside what is kept, and strips of several tiles in
the first product (GPU)."""
import math
import re

import pytest
import torch

import combine_router_softmax_top_gb300 as moe
from oracle import fp4_oracle as Q
from test_fp4_gpu import BF, experts, np8, run
from test_fp4_source_cpu import code

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from combine_router_softmax_top_gb300 import build
    build.build()


@pytest.mark.parametrize("T,E,k,F", [(4, 8, 2, 448), (200, 3, 2, 448), (7, 4, 2, 64), (300, 2, 2, 320)])
def test_the_scale_bytes_of_h_do_not_depend_on_what_is_kept(T, E, k, F):
    """Every block's byte (those past a row's blocks are unspecified)."""
    N, seen = T * k, []
    for keep in ((False, False), (True, True), (True, False), (False, True)):
        d, f, off, _, a, h, o, ws = experts(T, 320, E, k, F, 1, True)
        f.hs.fill_(0x5A)
        run(d, f, off, a if keep[0] else None, h if keep[1] else None, o, ws)
        assert moe.moe_device_status(d, ws) == moe.MOE_OK
        seen.append((Q.ungroup(np8(f.hs), N, F // 32), f.hq.clone(), o.clone()))
    for b, q, o in seen[1:]:
        assert (b == seen[0][0]).all() and torch.equal(q, seen[0][1]) and torch.equal(o, seen[0][2])


def strips(T, H, E, k, F):
    """Tiles of a strip in both products, by grouped_gemm_fp4.cu's rule; pairs: two SMs each."""
    want = [int(v) for v in re.search(r"kStrips\[2\] = \{(\d+), (\d+)\}", code("grouped_gemm_fp4.cu")).groups()]
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    row_tiles = max(1, T * k // 256)
    out = []
    for tiles, stages, n in ((-(-F // 128), -(-H // 256), want[0]), (-(-H // 256), -(-F // 256), want[1])):
        longest = max(-(-H // 256), -(-F // 256))
        slots = max(longest, 4) if longest <= 8 else 6
        across = min(tiles, math.ceil(n * pairs / row_tiles))
        out.append(1 if stages > slots else math.ceil(tiles / across))
    return out


@pytest.mark.parametrize("T,H,E,k,F,first,second", [(12800, 1088, 5, 2, 704, 3, 2), (30000, 1088, 5, 2, 704, 6, 3),
                                                    (24000, 128, 7, 3, 128, 1, 1), (9000, 512, 3, 2, 896, 3, 1),
                                                    (20000, 64, 2, 2, 2240, 18, 1)])
def test_strips(T, H, E, k, F, first, second):
    """Tiles side by side that share a strip's rows, against the same rows one expert and 1500 rows at
    a time (strips of one tile). The expected lengths are stated for 152 SMs."""
    if torch.cuda.get_device_properties(0).multi_processor_count == 152:
        assert strips(T, H, E, k, F) == [first, second]
    d, f, off, off_np, a, h, o, ws = experts(T, H, E, k, F, 1, False)
    run(d, f, off, a, h, o, ws)
    assert moe.moe_device_status(d, ws) == moe.MOE_OK
    again = o.clone()
    run(d, f, off, a, h, o, ws)
    assert torch.equal(again, o)
    for e in range(E):
        lo, hi = int(off_np[e]), int(off_np[e + 1])
        for r in range(lo, hi - 64, 1500):  # (64 rows or fewer are the other kernel's)
            n = hi - r if hi - r < 1500 + 64 else 1500
            de = moe.LayerDesc.of(n, H, 1, 1, F)
            fe = moe.Fp4Buffers(de)
            fe.xq.copy_(f.xq[r:r + n])
            fe.xs[:, :n].copy_(f.xs[:, r:r + n])
            oe = torch.zeros(n, H, dtype=BF, device="cuda")
            moe.moe_expert_ffn_fwd_fp4(de, fe.xq, fe.xs, torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                                       f.w1q[e].contiguous(), f.w1s[e].contiguous(), f.w2q[e].contiguous(),
                                       f.w2s[e].contiguous(), None, None, fe.hq, fe.hs, oe, ws)
            assert torch.equal(oe, o[r:r + n]), (e, r)
