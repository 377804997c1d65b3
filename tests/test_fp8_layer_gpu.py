"""The 8-bit layer calls: their outputs from their own 8-bit stages in float64, and calls from two
host threads.

Bounds, element by element. A sum of n products in fp32, in any order and with additions that may
truncate, is off by at most n 2^-23 sum |terms|; a rounding to bf16 by 2^-8 of the value. The
router's dz_j = g_j (dg_j - sum_l g_l dg_l) takes k + 3 fp32 operations, each off by at most 2^-23
of g_j (|dg_j| + sum_l g_l |dg_l|).
"""
import threading

import numpy as np
import pytest
import torch

import combine_router_softmax_top_gb300 as moe
import moe_synth
from test_fp8_gpu import LAYERS, np64

pytestmark = pytest.mark.gpu

B16, U = 2.0 ** -8, 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def built():
    from combine_router_softmax_top_gb300 import build
    build.build()
    torch.cuda.init()


def within(name, got, ref, tol):
    worst = float((np.abs(got - ref) / (tol + 2.0 ** -134)).max())
    assert np.isfinite(got).all() and worst <= 1, f"{name}: {worst:.3f} of the bound"


def layer(**shape):
    inp = moe_synth.make_inputs(**shape)
    d = moe.LayerDesc.of(**inp.shape_dict())
    b, q = moe.LayerBuffers(d), moe.Fp8Buffers(d)
    b.load_inputs(inp)
    q.quantize_weights(b.w1, b.w2)
    return d, b, q


@pytest.mark.parametrize("name", sorted(LAYERS))
def test_layer_outputs_follow_from_its_stages(name):
    d, b, q = layer(**LAYERS[name])
    moe.moe_layer_forward_fp8(d, b, q)
    moe.moe_layer_backward_fp8(d, b, q)
    assert moe.moe_device_status(d, b.ws) == moe.MOE_OK
    T, H, E, k, F = d.T, d.H, d.E, d.k, d.F
    slot, idx, off = (t.cpu().numpy() for t in (b.slot, b.idx, b.off))
    g, dg = np64(b.gates), np64(b.dgates)
    terms = g[:, :, None] * np64(b.o)[slot]
    y = terms.sum(1)
    within("y", np64(b.y), y, B16 * np.abs(y) + (1 + B16) * k * U * np.abs(terms).sum(1))
    # router
    x, w_r = np64(b.x), np64(b.w_r)
    gdg = (g * dg).sum(1, keepdims=True)
    dz, err = np.zeros((T, E)), np.zeros((T, E))
    np.put_along_axis(dz, idx, g * (dg - gdg), 1)
    np.put_along_axis(err, idx, (k + 3) * U * g * (np.abs(dg) + np.abs(g * dg).sum(1, keepdims=True)), 1)
    paths = np64(b.dx_perm)[slot]
    dx = paths.sum(1) + dz @ w_r
    size = np.abs(paths).sum(1) + np.abs(dz) @ np.abs(w_r)
    within("dx", np64(b.dx), dx,
           B16 * np.abs(dx) + (1 + B16) * (2 * k * U * size + err @ np.abs(w_r)))
    # (a sum over at most T tokens, by chunks; T 2^-23 bounds any order)
    within("dw_r", np64(b.dw_r), dz.T @ x, (T + 1) * U * np.abs(dz).T @ np.abs(x) + err.T @ np.abs(x))
    # weight gradients, from the bf16 rows
    rows = {n: np64(getattr(b, n)) for n in ("x_perm", "h", "d_o", "da")}
    dw1, dw2 = np64(b.dw1), np64(b.dw2)
    for e in range(E):
        s = slice(off[e], off[e + 1])
        n = int(off[e + 1] - off[e])
        for what, got, left, right in (("dw1", dw1[e], rows["da"][s], rows["x_perm"][s]),
                                       ("dw2", dw2[e], rows["d_o"][s], rows["h"][s])):
            ref = left.T @ right
            within(f"{what}[{e}]", got, ref,
                   B16 * np.abs(ref) + (1 + B16) * n * U * np.abs(left).T @ np.abs(right))


@pytest.mark.parametrize("T", [64, 1500])
def test_two_host_threads(T):
    """Two layers, each from a thread with a stream of its own: the backwards share the device's
    side stream. The same bits as alone."""
    layers = [layer(T=T, H=256, E=16, k=4, F=320, seed=s) for s in (61, 62)]
    names = ("y", "dx", "dw_r", "dw1", "dw2")

    def step(d, b, q):
        moe.moe_layer_forward_fp8(d, b, q)
        moe.moe_layer_backward_fp8(d, b, q)

    want = []
    for d, b, q in layers:
        step(d, b, q)
        want.append([getattr(b, n).clone() for n in names])
    torch.cuda.synchronize()
    meet, failed = threading.Barrier(2), []

    def work(i):
        try:
            d, b, q = layers[i]
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                meet.wait(60)
                for _ in range(15):
                    for n in names:
                        getattr(b, n).zero_()
                    step(d, b, q)
                    stream.synchronize()
                    for n, w in zip(names, want[i]):
                        assert torch.equal(getattr(b, n), w), n
        except BaseException as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not failed, failed
    for d, b, _ in layers:
        assert moe.moe_device_status(d, b.ws) == moe.MOE_OK
