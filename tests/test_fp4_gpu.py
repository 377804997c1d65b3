"""The 4-bit experts on the GPU against the float64 oracle, stage by stage: each stage is
run by the oracle on the GPU's own inputs of that stage.

Bounds. Products of e2m1 values with power-of-two scales are exact in fp32, so an element of a
product differs from the oracle's by the fp32 summation alone, in any order: K 2^-24 sum |x w|
(twice that where the order's partial sums are rounded by truncation: the bounds use 2 K 2^-24),
plus half a bf16 step where it is stored as bf16. h = silu(g) u is fp32 with a sigmoid of
relative error 7e-6 at most, and |silu'| <= 1.1."""
import threading

import numpy as np
import pytest
import torch

import combine_router_softmax_top_gb300 as moe
from oracle import fp4_oracle as Q

pytestmark = pytest.mark.gpu
BF, U8 = torch.bfloat16, torch.uint8


@pytest.fixture(scope="module", autouse=True)
def built():
    from combine_router_softmax_top_gb300 import build
    build.build()


def f64(t):
    return t.detach().double().cpu().numpy()


def np8(t):
    return t.detach().cpu().numpy()


def rnd(*s, std=1.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*s, generator=g, device="cuda") * std).to(BF)


def routing(T, E, k, skew, seed):
    """slot [T, k], off [E + 1]; skew 0: even, 1: a few experts take most, 2: one takes all it can."""
    rng = np.random.default_rng(seed)
    if skew == 0:
        idx = (k * np.arange(T)[:, None] + np.arange(k)) % E
    elif skew == 1:
        z = rng.standard_normal((T, E)) + 4.0 / (1 + np.arange(E))
        idx = np.argsort(-z, 1)[:, :k]
    else:
        idx = np.tile(np.arange(k) + E - k, (T, 1))
    cnt = np.bincount(idx.ravel(), minlength=E)
    off = np.concatenate([[0], cnt.cumsum()])
    slot = np.empty(T * k, np.int64)
    slot[np.argsort(idx.ravel(), kind="stable")] = np.arange(T * k)
    to = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    return to(slot.reshape(T, k)), to(off), off


def weights(f, E, F, H):
    """The values of quantised weights as the library holds them."""
    w1 = Q.values(Q.unpack(np8(f.w1q)).reshape(E, 2, F, H), Q.ungroup(np8(f.w1s), F, H // 32))
    w2 = Q.values(Q.unpack(np8(f.w2q)), Q.ungroup(np8(f.w2s), H, F // 32))
    return w1.reshape(E, 2 * F, H), w2


# ----------------------------------------------------------------------------- weights
@pytest.mark.parametrize("E,H,F", [(1, 64, 64), (3, 320, 192), (2, 256, 448), (4, 576, 64),
                                   (5, 128, 512), (2, 2048, 768)])
@pytest.mark.parametrize("keep", [False, True])
def test_weights(E, H, F, keep):
    d = moe.LayerDesc.of(4, H, E, 1, F)
    f = moe.Fp4Buffers(d)
    w1, w2 = rnd(E, 2 * F, H, std=0.02, seed=1), rnd(E, H, F, std=0.02, seed=2)
    w1[0, 0, :32] = 0
    w1[0, 1, :32] = -0.0
    w2[0, 0, :8] = torch.tensor([6, -6, 5, -5, 2.5, 0.25, 0.75, -3.5], device="cuda").to(BF)
    w2[-1, -1, -32:] = torch.arange(32, device="cuda").to(BF) * 2.0 ** -133  # subnormals
    w1[-1, -1, -32:] = 3.3895313892515355e38
    v = (torch.full_like(w1, 7.0), torch.full_like(w2, 7.0)) if keep else (None, None)
    f.w1s.fill_(9), f.w2s.fill_(9)
    f.quantize_weights(w1, w2, *v)
    for w, q, s, R in ((w1.view(E, 2, F, H), f.w1q, f.w1s, F), (w2, f.w2q, f.w2s, H)):
        c, b = Q.quantize(f64(w))
        assert (np8(q).reshape(*c.shape[:-1], -1) == Q.pack(c)).all()
        assert (np8(s) == Q.groups(b)).all()  # the bytes past the last block are 0
    if keep:
        # 3.39e38 = 3.98 2^126 rounds to 4 2^126 = 2^128, which bf16 holds as an infinity
        for got, want in zip(v, weights(f, E, F, H)):
            assert (f64(got) == np.where(np.abs(want) == 2.0 ** 128, np.copysign(np.inf, want), want)).all()


def test_weights_in_place_and_not_finite():
    E, H, F = 2, 192, 128
    d = moe.LayerDesc.of(4, H, E, 1, F)
    f, g = moe.Fp4Buffers(d), moe.Fp4Buffers(d)
    w1, w2 = rnd(E, 2 * F, H, seed=1), rnd(E, H, F, seed=2)
    f.quantize_weights(w1, w2)
    a1, a2 = w1.clone(), w2.clone()
    g.quantize_weights(a1, a2, a1, a2)
    assert torch.equal(f.w1q, g.w1q) and torch.equal(f.w2s, g.w2s)
    v1, v2 = weights(f, E, F, H)
    assert (f64(a1) == v1).all() and (f64(a2) == v2).all()
    w1[0, 3, 40], w1[1, 7, 64], w2[0, 1, 0] = float("nan"), float("inf"), -float("inf")
    f.quantize_weights(w1, w2, a1, a2)
    b1, b2 = Q.ungroup(np8(f.w1s), F, H // 32), Q.ungroup(np8(f.w2s), H, F // 32)
    assert b1[0, 0, 3, 1] == 255 and b1[1, 0, 7, 2] == 255 and b2[0, 1, 0] == 255
    assert (b1 == 255).sum() == 2 and (b2 == 255).sum() == 1
    assert torch.isnan(a1[0, 3, 32:64]).all() and torch.isnan(a1).sum() == 64


# ----------------------------------------------------------------------------- permute
@pytest.mark.parametrize("T,H,k", [(1, 64, 1), (1, 2048, 8), (3, 320, 2), (33, 576, 5), (7, 4096, 3),
                                   (129, 192, 32), (500, 1024, 4)])
def test_permute(T, H, k):
    E, N = 40, T * k
    d = moe.LayerDesc.of(T, H, E, k, 64)
    slot, _, _ = routing(T, E, k, 1, T)
    x = rnd(T, H, seed=3) * torch.exp(2 * rnd(T, 1, seed=4))
    x[0, :32] = 0
    f = moe.Fp4Buffers(d)
    f.xq.fill_(0x5A), f.xs.fill_(0x5A)
    if N > 3:  # slots out of range are skipped, their rows left as they were
        slot.view(-1)[1], slot.view(-1)[2] = -1, N + 5
    moe.moe_permute_fp4(d, x, slot, f.xq, f.xs)
    c, b = Q.quantize(f64(x))
    q, s = np.full((N, H // 2), 0x5A, np.uint8), np.full(tuple(f.xs.shape), 0x5A, np.uint8)
    packed, grp = Q.pack(c), Q.groups(b)
    for t, row in enumerate(slot.tolist()):
        for r in row:
            if 0 <= r < N:
                q[r], s[:, r] = packed[t], grp[:, t]
    assert (np8(f.xq) == q).all() and (np8(f.xs) == s).all()


# ----------------------------------------------------------------------------- experts
def experts(T, H, E, k, F, skew, keep, seed=0, stream=None, x=None):
    d = moe.LayerDesc.of(T, H, E, k, F)
    N = T * k
    f = moe.Fp4Buffers(d)
    f.quantize_weights(rnd(E, 2 * F, H, std=0.3 / H ** 0.5 * 8, seed=seed + 1),
                       rnd(E, H, F, std=0.02, seed=seed + 2))
    slot, off, off_np = routing(T, E, k, skew, seed)
    moe.moe_permute_fp4(d, rnd(T, H, seed=seed + 3) if x is None else x, slot, f.xq, f.xs)
    pad = lambda c: torch.full((N + 2, c), 3.0, dtype=BF, device="cuda")  # noqa: E731
    a, h, o = (pad(2 * F), pad(F), pad(H)) if keep else (None, None, pad(H))
    ws = torch.zeros(moe.moe_workspace_size(d), dtype=U8, device="cuda")
    f.hq.fill_(0x11)
    return d, f, off, off_np, a, h, o, ws


def run(d, f, off, a, h, o, ws, stream=None):
    moe.moe_expert_ffn_fwd_fp4(d, f.xq, f.xs, off, f.w1q, f.w1s, f.w2q, f.w2s, a, h, f.hq, f.hs, o,
                               ws, stream)


def half_ulp(v):
    """Half a bf16 step at v."""
    return np.abs(v) * 2.0 ** -8


def check(d, f, off, a, h, o, ws):
    """The stages' outputs against the oracle's on the GPU's own inputs."""
    assert moe.moe_device_status(d, ws) == moe.MOE_OK
    E, H, F, N = d.E, d.H, d.F, d.T * d.k
    used = int(off[-1])
    w1, w2 = weights(f, E, F, H)
    x = Q.values(Q.unpack(np8(f.xq)), Q.ungroup(np8(f.xs), N, H // 32))
    A = Q.grouped(x, off, w1)
    eA = 2 * H * 2.0 ** -24 * Q.grouped(np.abs(x), off, np.abs(w1))
    g, u = np.split(A, 2, axis=1)
    eg, eu = np.split(eA, 2, axis=1)
    H1 = Q.swiglu(A)
    eH = 1.1 * eg * (np.abs(u) + eu) + np.abs(g) * Q.sigmoid(g) * eu + 8e-6 * np.abs(H1) + 1e-37
    if a is not None:
        av, hv = f64(a), f64(h)
        assert (av[used:] == 3).all() and (hv[used:] == 3).all()
        assert (np.abs(av[:used] - A[:used]) <= (eA + half_ulp(np.abs(A) + eA))[:used]).all()
        assert (np.abs(hv[:used] - H1[:used]) <= (eH + half_ulp(np.abs(H1) + eH))[:used]).all()
    # h in 4 bits: the scale byte is the oracle's of a maximum within the error, each value the
    # nearest one up to the error
    c, b = Q.unpack(np8(f.hq)), Q.ungroup(np8(f.hs), N, F // 32)
    lo = np.abs(H1) - eH
    blocks = lambda v: v.reshape(N, -1, 32).max(-1)  # noqa: E731
    assert (b[:used] >= Q.scale_byte(np.maximum(blocks(lo), 0))[:used]).all()
    assert (b[:used] <= Q.scale_byte(blocks(np.abs(H1) + eH))[:used]).all()
    hs = np.repeat(Q.scale(np.where(b > 254, 0, b)), 32, axis=1)
    hv = Q.of_codes(c) * hs
    step = hs * np.array([.5, .5, .5, .5, 1, 1, 2, 2])[c & 7]  # (the step above a value is the wider one)
    assert (np.abs(hv - H1)[:used] <= (step / 2 + eH)[:used]).all()
    O = Q.grouped(hv, off, w2)  # noqa: E741
    eO = 2 * F * 2.0 ** -24 * Q.grouped(np.abs(hv), off, np.abs(w2))
    ov = f64(o)
    assert (ov[used:] == 3).all()
    assert (np.abs(ov[:used] - O[:used]) <= (eO + half_ulp(np.abs(O) + eO) + 1e-40)[:used]).all()
    assert used == 0 or np.abs(ov[:used]).max() > 0


SHAPES = [  # T, H, E, k, F, skew
    (1, 64, 1, 1, 64, 0), (1, 128, 4, 2, 64, 0), (1, 256, 8, 8, 320, 0), (2, 320, 3, 1, 448, 0),
    (5, 192, 16, 4, 192, 1), (33, 576, 2, 1, 64, 0), (64, 512, 32, 8, 256, 1), (40, 64, 2, 2, 704, 2),
    (31, 1344, 5, 3, 128, 1), (96, 256, 200, 2, 128, 1), (48, 2048, 1, 1, 192, 0),
    # many rows an expert on average
    (49, 64, 1, 1, 64, 0), (100, 320, 2, 1, 448, 0), (129, 192, 2, 2, 64, 0), (257, 256, 2, 2, 320, 1),
    (400, 512, 8, 4, 192, 1), (600, 64, 3, 2, 576, 1), (500, 576, 6, 3, 256, 2), (1000, 320, 16, 4, 448, 1),
    (255, 1344, 4, 2, 128, 1), (3000, 128, 4, 2, 128, 1), (64, 2048, 1, 1, 768, 0),
    (300, 2304, 2, 1, 64, 0), (300, 64, 2, 1, 2304, 0), (290, 2624, 1, 1, 2112, 0), (70, 64, 1, 1, 2048, 0),
    (3, 16384, 2, 1, 64, 0), (70, 16384, 1, 1, 64, 0), (70, 64, 1, 1, 16384, 0), (5, 64, 256, 32, 64, 1),
    (65, 64, 1, 1, 64, 0), (70, 2048, 1, 1, 768, 0), (140, 320, 2, 1, 448, 0), (128, 64, 2, 2, 192, 2),
]


@pytest.mark.parametrize("T,H,E,k,F,skew", SHAPES)
@pytest.mark.parametrize("keep", [False, True])
def test_experts(T, H, E, k, F, skew, keep):
    d, f, off, off_np, a, h, o, ws = experts(T, H, E, k, F, skew, keep, seed=T + H)
    run(d, f, off, a, h, o, ws)
    check(d, f, off_np, a, h, o, ws)


@pytest.mark.parametrize("T,E,k", [(4, 8, 2), (200, 3, 2)])
def test_what_is_kept_changes_nothing(T, E, k):
    outs = []
    for keep in (False, True):
        d, f, off, off_np, a, h, o, ws = experts(T, 320, E, k, 448, 1, keep)
        run(d, f, off, a, h, o, ws)
        outs.append((o, f.hq.clone(), f.hs[..., :7].clone()))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    kept = h
    d, f, off, off_np, a, h, o, ws = experts(T, 320, E, k, 448, 1, True)
    run(d, f, off, a, None, o, ws)
    assert torch.equal(o, outs[0][0]) and (h == 3).all()
    run(d, f, off, None, h, o, ws)
    assert torch.equal(o, outs[0][0]) and torch.equal(h, kept)


@pytest.mark.parametrize("T,E,k", [(6, 8, 2), (300, 2, 2)])
def test_rows_past_the_experts_and_bad_offsets(T, E, k):
    d, f, off, off_np, a, h, o, ws = experts(T, 192, E, k, 128, 0, True)
    N = T * k
    off_np = np.minimum(off_np, N - 5)  # the last rows belong to nobody
    run(d, f, torch.tensor(off_np, dtype=torch.int32, device="cuda"), a, h, o, ws)
    check(d, f, off_np, a, h, o, ws)
    # outside 0..N: taken as the nearest bound
    d, f, off, off_np, a, h, o, ws = experts(T, 192, E, k, 128, 0, True)
    bad = off.clone()
    bad[0], bad[-1] = -7, N + 900
    run(d, f, bad, a, h, o, ws)
    check(d, f, off_np, a, h, o, ws)
    # no rows at all
    o.fill_(3)
    run(d, f, torch.zeros_like(off), None, None, o, ws)
    assert (o == 3).all() and moe.moe_device_status(d, ws) == moe.MOE_OK


@pytest.mark.parametrize("T,E,k", [(6, 4, 2), (300, 2, 2)])
def test_a_row_that_is_not_finite_stays_alone(T, E, k):
    x = rnd(T, 192, seed=9)
    d, f, off, off_np, a, h, o, ws = experts(T, 192, E, k, 128, 0, True, x=x)
    run(d, f, off, a, h, o, ws)
    want = o.clone()
    x[1, 70], x[3, 0] = float("nan"), float("inf")
    d, f, off, off_np, a, h, o, ws = experts(T, 192, E, k, 128, 0, True, x=x)
    run(d, f, off, a, h, o, ws)
    slot = routing(T, E, k, 0, 0)[0].long()
    bad = slot[[1, 3]].flatten()
    assert torch.isnan(o[bad]).all()
    good = torch.ones(T * k + 2, dtype=torch.bool, device="cuda")
    good[bad] = False
    assert torch.equal(o[good], want[good])


@pytest.mark.parametrize("T,E,k", [(6, 4, 2), (300, 2, 2)])
def test_a_weight_that_is_not_finite_stays_in_its_expert(T, E, k):
    d, f, off, off_np, a, h, o, ws = experts(T, 192, E, k, 128, 0, True)
    run(d, f, off, a, h, o, ws)
    want = o.clone()
    w1 = rnd(E, 256, 192, std=0.3 / 192 ** 0.5 * 8, seed=1)
    w1[1, 3, 5] = float("nan")
    f.quantize_weights(w1, rnd(E, 192, 128, std=0.02, seed=2))
    run(d, f, off, a, h, o, ws)
    lo, hi = off_np[1], off_np[2]
    assert torch.isnan(a[lo:hi, 3]).all() and torch.isnan(a[:-2].float()).sum() == hi - lo
    assert torch.isnan(o[lo:hi]).all()
    assert torch.equal(o[:lo], want[:lo]) and torch.equal(o[hi:], want[hi:])


@pytest.mark.parametrize("T,E,k,F", [(20, 16, 4, 192), (4000, 4, 2, 256)])
def test_streams_and_captures(T, E, k, F):
    """Chains on two streams at once, each with its workspace, and replays of a capture."""
    sets = [experts(T, 256, E, k, F, 1, False, seed=s) for s in (1, 50)]
    alone = []
    for d, f, off, _, a, h, o, ws in sets:
        run(d, f, off, a, h, o, ws)
        alone.append(o.clone())
        o.fill_(3)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        for st, (d, f, off, _, a, h, o, ws) in zip(streams, sets):
            run(d, f, off, a, h, o, ws, st)
    torch.cuda.synchronize()
    for want, (d, _, _, _, _, _, o, ws) in zip(alone, sets):
        assert torch.equal(o, want) and moe.moe_device_status(d, ws) == moe.MOE_OK
        o.fill_(3)
    d, f, off, _, a, h, o, ws = sets[0]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(d, f, off, a, h, o, ws)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, alone[0]) and moe.moe_device_status(d, ws) == moe.MOE_OK


@pytest.mark.parametrize("T,H,E,k,F", [(24000, 128, 7, 3, 128), (30000, 1088, 5, 2, 704)])
def test_many_tiles_a_pair(T, H, E, k, F):
    """Many tiles for each CTA pair (in strips of one, in strips of three), experts of every
    size in turn."""
    d, f, off, off_np, a, h, o, ws = experts(T, H, E, k, F, 1, False)
    run(d, f, off, a, h, o, ws)
    assert moe.moe_device_status(d, ws) == moe.MOE_OK
    first = o.clone()
    for _ in range(3):
        run(d, f, off, a, h, o, ws)
        assert torch.equal(first, o)
    # the same rows in small batches, an expert at a time
    for e in range(E):
        lo, hi = int(off_np[e]), int(off_np[e + 1])
        for r in range(lo, hi, 1500):
            n = min(1500, hi - r)
            de = moe.LayerDesc.of(n, H, 1, 1, F)
            fe = moe.Fp4Buffers(de)
            fe.xq.copy_(f.xq[r:r + n])
            fe.xs[:, :n].copy_(f.xs[:, r:r + n])
            oe = torch.zeros(n, H, dtype=BF, device="cuda")
            moe.moe_expert_ffn_fwd_fp4(de, fe.xq, fe.xs, torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                                       f.w1q[e].contiguous(), f.w1s[e].contiguous(), f.w2q[e].contiguous(),
                                       f.w2s[e].contiguous(), None, None, fe.hq, fe.hs, oe, ws)
            assert torch.equal(oe, o[r:r + n]), (e, r)


def test_buffers_past_32_bits():
    """Outputs of more than 2^32 bytes and activations of more than 2^31 elements."""
    T, H, E, k, F = 1100000, 2048, 2, 1, 64
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB of device memory")
    d = moe.LayerDesc.of(T, H, E, k, F)
    f = moe.Fp4Buffers(d)
    f.quantize_weights(rnd(E, 2 * F, H, std=0.05, seed=1), rnd(E, H, F, std=0.05, seed=2))
    tail = rnd(700, H, seed=3)
    x = torch.zeros(T, H, dtype=BF, device="cuda")
    x[-700:] = tail
    slot = torch.arange(T, dtype=torch.int32, device="cuda")
    moe.moe_permute_fp4(d, x, slot, f.xq, f.xs)
    o = torch.full((T, H), 3.0, dtype=BF, device="cuda")
    ws = torch.zeros(moe.moe_workspace_size(d), dtype=U8, device="cuda")
    off = torch.tensor([0, 5, T], dtype=torch.int32, device="cuda")
    run(d, f, off, None, None, o, ws)
    assert moe.moe_device_status(d, ws) == moe.MOE_OK
    assert (o[5:1000] == 0).all() and (o[-2000:-700] == 0).all()
    d2 = moe.LayerDesc.of(700, H, E, k, F)
    f2 = moe.Fp4Buffers(d2, weights=f)
    moe.moe_permute_fp4(d2, tail, slot[:700], f2.xq, f2.xs)
    o2 = torch.zeros(700, H, dtype=BF, device="cuda")
    run(d2, f2, torch.tensor([0, 0, 700], dtype=torch.int32, device="cuda"), None, None, o2, ws)
    assert torch.equal(o[-700:], o2)


# ----------------------------------------------------------------------------- the layer
@pytest.mark.parametrize("T,E,k", [(1, 16, 4), (37, 16, 4), (900, 8, 2), (300, 200, 3)])
def test_layer_forward(T, E, k):
    """The layer call is its stages, serving and saving."""
    H, F = 256, 192
    d = moe.LayerDesc.of(T, H, E, k, F)
    b = moe.LayerBuffers(d)
    b.x.copy_(rnd(T, H, seed=1))
    b.w_r.copy_(rnd(E, H, std=0.1, seed=2))
    w1, w2 = rnd(E, 2 * F, H, std=0.1, seed=3), rnd(E, H, F, std=0.1, seed=4)
    f = moe.Fp4Buffers(d)
    f.quantize_weights(w1, w2)
    moe.moe_layer_forward_fp4(d, b, f, save=False)
    assert moe.moe_device_status(d, b.ws) == moe.MOE_OK
    y = b.y.clone()
    moe.moe_layer_forward_fp4(d, b, f, save=True)
    assert torch.equal(y, b.y) and b.h.abs().max() > 0
    assert torch.equal(b.x_perm[b.slot.long()], b.x[:, None].expand(T, k, H))
    g = moe.Fp4Buffers(d, weights=f)
    moe.moe_permute_fp4(d, b.x, b.slot, g.xq, g.xs)
    o = torch.zeros_like(b.o)
    run(d, g, b.off, None, None, o, b.ws)
    assert torch.equal(o, b.o)
    moe.moe_combine(d, o, b.slot, b.gates, b.y)
    assert torch.equal(y, b.y)


@pytest.mark.parametrize("T,E,k", [(5, 4, 2), (260, 4, 2)])
def test_training_through_the_layer(T, E, k):
    """moe_layer_backward on the values of the 4-bit weights: the gradient of the forward
    with its roundings passed through, in float64 from the GPU's own saved tensors."""
    H, F = 128, 192
    N = T * k
    d = moe.LayerDesc.of(T, H, E, k, F)
    b = moe.LayerBuffers(d)
    b.x.copy_(rnd(T, H, seed=1))
    b.dy.copy_(rnd(T, H, seed=5))
    b.w_r.copy_(rnd(E, H, std=0.1, seed=2))
    f = moe.Fp4Buffers(d)
    f.quantize_weights(rnd(E, 2 * F, H, std=0.1, seed=3), rnd(E, H, F, std=0.1, seed=4), b.w1, b.w2)
    moe.moe_layer_forward_fp4(d, b, f, save=True)
    moe.moe_layer_backward(d, b)
    assert moe.moe_device_status(d, b.ws) == moe.MOE_OK
    w1, w2 = weights(f, E, F, H)
    assert (f64(b.w1) == w1).all()
    off = np8(b.off)
    a, d_o = f64(b.a), f64(b.d_o)
    dh = Q.grouped(d_o, off, np.swapaxes(w2, 1, 2))
    edh = 2 * H * 2.0 ** -24 * Q.grouped(np.abs(d_o), off, np.abs(np.swapaxes(w2, 1, 2)))
    g, u = np.split(a, 2, axis=1)
    s = Q.sigmoid(g)
    fac = np.concatenate([u * s * (1 + g * (1 - s)), g * s], 1)
    da = np.concatenate([dh, dh], 1) * fac
    eda = np.concatenate([edh, edh], 1) * np.abs(fac) + 2e-5 * np.abs(da) + 1e-5 * np.abs(np.concatenate([dh * u, dh * g], 1))
    gda = f64(b.da)
    assert (np.abs(gda - da) <= eda + half_ulp(np.abs(da) + eda) + 1e-37).all()
    dxp = Q.grouped(gda, off, np.swapaxes(w1, 1, 2))
    e = 4 * F * 2.0 ** -24 * Q.grouped(np.abs(gda), off, np.abs(np.swapaxes(w1, 1, 2)))
    assert (np.abs(f64(b.dx_perm) - dxp) <= e + half_ulp(np.abs(dxp) + e) + 1e-37).all()
    h = f64(b.h)
    for i in range(E):
        lo, hi = off[i], off[i + 1]
        for got, l, r in ((b.dw1, gda, f64(b.x_perm)), (b.dw2, d_o, h)):
            want, mag = l[lo:hi].T @ r[lo:hi], np.abs(l[lo:hi]).T @ np.abs(r[lo:hi])
            e = 2 * max(hi - lo, 1) * 2.0 ** -24 * mag
            assert (np.abs(f64(got[i]) - want) <= e + half_ulp(np.abs(want) + e) + 1e-37).all()


def test_refuses_wrong_tensors():
    d, f, off, _, a, h, o, ws = experts(4, 128, 2, 1, 64, 0, False)
    args = [f.xq, f.xs, off, f.w1q, f.w1s, f.w2q, f.w2s, None, None, f.hq, f.hs, o, ws]
    for i, bad, why in ((0, f.xq[:1], "fewer"), (1, f.xs[:, :2], "contiguous|fewer"), (2, off.long(), "int64"),
                        (4, f.w1s[:1], "fewer"), (3, f.w1q.cpu(), "device"), (9, f.hq.t(), "contiguous"),
                        (10, None, "None"), (11, o.float(), "float32")):
        with pytest.raises(moe.MoeError, match=why):
            moe.moe_expert_ffn_fwd_fp4(d, *[bad if j == i else t for j, t in enumerate(args)])


@pytest.mark.parametrize("T,E,k", [(9, 16, 4), (700, 4, 2)])
def test_layer_forward_captured(T, E, k):
    """A captured serving forward, replayed on new inputs, with bf16 work of the same
    workspace between the replays."""
    H, F = 256, 192
    d = moe.LayerDesc.of(T, H, E, k, F)
    b = moe.LayerBuffers(d)
    b.w_r.copy_(rnd(E, H, std=0.1, seed=2))
    b.w1.copy_(rnd(E, 2 * F, H, std=0.1, seed=3))
    b.w2.copy_(rnd(E, H, F, std=0.1, seed=4))
    f = moe.Fp4Buffers(d)
    f.quantize_weights(b.w1, b.w2)
    want = []
    for seed in (1, 2, 3):
        b.x.copy_(rnd(T, H, seed=seed))
        moe.moe_layer_forward_fp4(d, b, f)
        want.append(b.y.clone())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_layer_forward_fp4(d, b, f)
    for seed, y in zip((1, 2, 3), want):
        b.x.copy_(rnd(T, H, seed=seed))
        moe.moe_layer_forward(d, b)
        b.y.zero_()
        g.replay()
        assert torch.equal(b.y, y)
    assert moe.moe_device_status(d, b.ws) == moe.MOE_OK


def test_two_host_threads():
    """Calls from two threads, each on its stream with its workspace, and each the first CUDA
    call of its thread (the driver's map encoder wants a context, which the thread lacks)."""
    sets = [experts(T, 256, 8, 2, 320, 1, False, seed=T) for T in (12, 900)]
    want = []
    for d, f, off, _, a, h, o, ws in sets:
        run(d, f, off, a, h, o, ws)
        want.append(o.clone())
        o.fill_(3)
    torch.cuda.synchronize()
    errors = []

    def work(s, w):
        try:
            st = torch.cuda.Stream()
            d, f, off, _, a, h, o, ws = s
            for _ in range(50):
                run(d, f, off, a, h, o, ws, st)
            st.synchronize()
            assert torch.equal(o, w) and moe.moe_device_status(d, ws, st) == moe.MOE_OK
        except BaseException as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=p) for p in zip(sets, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_first_call_of_a_thread_in_bf16():
    """The same for the bf16 experts."""
    T, E, k, H, F = 40, 4, 2, 128, 64
    d = moe.LayerDesc.of(T, H, E, k, F)
    b = moe.LayerBuffers(d)
    b.x.copy_(rnd(T, H, seed=1)), b.w1.copy_(rnd(E, 2 * F, H, seed=2)), b.w2.copy_(rnd(E, H, F, seed=3))
    moe.moe_layer_forward(d, b)
    want, errors = b.o.clone(), []
    b.o.zero_()
    torch.cuda.synchronize()
    raw = torch.cuda.current_stream().cuda_stream

    def work():
        try:
            moe.moe_expert_ffn_fwd(d, b.x_perm, b.off, b.w1, b.w2, b.a, b.h, b.o, b.ws, raw)
        except BaseException as e:  # noqa: BLE001
            errors.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not errors and torch.equal(b.o, want), errors


@pytest.mark.parametrize("seed", range(12))
def test_seeded_shapes(seed):
    """Random shapes over the whole range, on both sides of the few-rows rule."""
    rng = np.random.default_rng(1000 + seed)
    H, F = (64 * int(rng.integers(1, 20)) for _ in range(2))
    E = int(rng.integers(1, 40))
    k = int(rng.integers(1, min(E, 8) + 1))
    T = int(np.exp(rng.uniform(0, np.log(1200))))
    d, f, off, off_np, a, h, o, ws = experts(T, H, E, k, F, int(rng.integers(0, 3)), bool(seed & 1), seed=seed)
    run(d, f, off, a, h, o, ws)
    check(d, f, off_np, a, h, o, ws)


def test_no_tokens():
    """A layer without tokens: nothing is written, nothing is wrong."""
    d = moe.LayerDesc.of(0, 128, 4, 2, 64)
    b, f = moe.LayerBuffers(d), moe.Fp4Buffers(d)
    f.quantize_weights(b.w1, b.w2)
    b.y.fill_(3), b.o.fill_(3)
    for save in (False, True):
        moe.moe_layer_forward_fp4(d, b, f, save=save)
    moe.moe_permute_fp4(d, b.x, b.slot, f.xq, f.xs)
    run(d, f, b.off, None, None, b.o, b.ws)
    assert moe.moe_device_status(d, b.ws) == moe.MOE_OK
    assert (b.y == 3).all() and (b.o == 3).all()
