"""What the gradient behind the 4-bit forward multiplies by (include/moe.h, "4-bit experts"): the
weights' gradients take x_perm and h in bf16, as kept, and not their 4-bit values.

Bounds: a sum of n exact products in fp32, in any order, errs by 2 n 2^-24 of the sum of their
magnitudes at most, and bf16 adds half a step."""
import numpy as np
import pytest
import torch

import combine_router_softmax_top_gb300 as moe
from oracle import fp4_oracle as Q
from test_fp4_gpu import f64, half_ulp, np8, rnd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from combine_router_softmax_top_gb300 import build
    build.build()


@pytest.mark.parametrize("T,E,k", [(6, 4, 2), (280, 4, 2)])
def test_weight_gradients_take_the_kept_rows(T, E, k):
    H, F = 128, 192
    N = T * k
    d = moe.LayerDesc.of(T, H, E, k, F)
    b, f = moe.LayerBuffers(d), moe.Fp4Buffers(d)
    b.x.copy_(rnd(T, H, seed=1))
    b.dy.copy_(rnd(T, H, seed=5))
    b.w_r.copy_(rnd(E, H, std=0.1, seed=2))
    f.quantize_weights(rnd(E, 2 * F, H, std=0.1, seed=3), rnd(E, H, F, std=0.1, seed=4), b.w1, b.w2)
    moe.moe_layer_forward_fp4(d, b, f, save=True)
    moe.moe_layer_backward(d, b)
    assert moe.moe_device_status(d, b.ws) == moe.MOE_OK
    off = np8(b.off)
    rounded = (Q.values(Q.unpack(np8(f.xq)), Q.ungroup(np8(f.xs), N, H // 32)),
               Q.values(Q.unpack(np8(f.hq)), Q.ungroup(np8(f.hs), N, F // 32)))
    apart = 0
    for e in range(E):
        rows = slice(off[e], off[e + 1])
        n = off[e + 1] - off[e]
        for got, left, kept, codes in ((b.dw1, f64(b.da), f64(b.x_perm), rounded[0]),
                                       (b.dw2, f64(b.d_o), f64(b.h), rounded[1])):
            want, other = left[rows].T @ kept[rows], left[rows].T @ codes[rows]
            bound = 2 * max(n, 1) * 2.0 ** -24 * (np.abs(left[rows]).T @ np.abs(kept[rows]))
            bound = bound + half_ulp(np.abs(want) + bound) + 1e-37
            assert (np.abs(f64(got[e]) - want) <= bound).all()
            apart += (np.abs(f64(got[e]) - other) > bound).sum()
    assert apart > 0, "the two readings are not told apart"
