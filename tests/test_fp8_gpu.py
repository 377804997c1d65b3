"""The 8-bit experts on the GPU against their float64 oracle.

What is held in 8 bits must match bit for bit (values and scale bytes), given
the same bf16 input. Products are compared stage by stage on the GPU's own
stage inputs, element by element. A stage's result v = bf16(s), s the fp32 sum:
  - rounding to bf16 is off by at most 2^-8 of the value;
  - s differs from the exact sum by at most K 2^-24 sum_k |a_k b_k| (the bound of
    K fp32 additions in any order; products of e4m3 values and powers of two are
    exact in fp32);
  - SwiGLU and its gradient add a few fp32 roundings and the fast exponential
    and division: 2^-20 of the value.
"""
import numpy as np
import pytest
import torch

import combine_router_softmax_top_gb300 as moe
import moe_synth
from oracle import fp8_oracle as O

pytestmark = pytest.mark.gpu

HALF16, U32, ELEM = 2.0 ** -8, 2.0 ** -24, 2.0 ** -20


@pytest.fixture(scope="module", autouse=True)
def built():
    from combine_router_softmax_top_gb300 import build
    build.build()
    torch.cuda.init()


def np64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def q64(t):
    """e4m3 tensor -> float64 values."""
    return t.detach().float().double().cpu().numpy()


def same(name, got, want):
    got, want = np.asarray(got), np.asarray(want)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    bad = ~((got == want) | (np.isnan(got) & np.isnan(want))) if got.dtype.kind == "f" else got != want
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size} differ, first at {np.argwhere(bad)[:3].tolist()}"


def close(name, got, ref, acc):
    """|got - ref| <= 2^-8 |ref| + (1 + 2^-8) acc, element by element (subnormal bf16: 2^-134)."""
    tol = HALF16 * np.abs(ref) + (1 + HALF16) * acc + 2.0 ** -134
    err = np.abs(got - ref)
    worst = float((err / tol).max()) if err.size else 0.0
    assert np.isfinite(got).all() and worst <= 1, f"{name}: {worst:.3f} of the bound"
    return worst


def routing(T, E, k, kind, seed):
    """(idx, gates, off, slot) of numpy-drawn choices."""
    rng = np.random.default_rng(seed)
    if kind == "balanced":
        idx = (k * np.arange(T)[:, None] + np.arange(k)) % E
    else:
        bias = 6.0 * rng.permutation(E) / max(E - 1, 1)
        idx = np.argsort(-(rng.standard_normal((T, E)) + bias), axis=1)[:, :k]
    gates = rng.random((T, k)).astype(np.float32) + 0.05
    gates /= gates.sum(1, keepdims=True)
    cnt = np.bincount(idx.ravel(), minlength=E)
    off = np.concatenate([[0], np.cumsum(cnt)])
    slot = np.empty(T * k, np.int64)
    slot[np.argsort(idx.ravel(), kind="stable")] = np.arange(T * k)
    return idx, gates, off, slot.reshape(T, k)


class Case:
    """One layer's inputs and buffers, from a seed."""

    def __init__(self, T, H, E, k, F, kind="skewed", seed=0, w_std=0.02, x=None):
        self.T, self.H, self.E, self.k, self.F, self.N = T, H, E, k, F, T * k
        self.d = moe.LayerDesc.of(T, H, E, k, F)
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(torch.bfloat16)  # noqa: E731
        self.x = (rnd(T, H) if x is None else x).cuda()
        self.dy = rnd(T, H).cuda()
        self.w1, self.w2 = rnd(E, 2 * F, H, std=w_std).cuda(), rnd(E, H, F, std=w_std).cuda()
        idx, gates, off, slot = routing(T, E, k, kind, seed)
        self.off_np, self.slot_np, self.gates_np = off, slot, gates
        i32 = lambda a: torch.from_numpy(a.astype(np.int32)).cuda()  # noqa: E731
        self.off, self.slot, self.gates = i32(off), i32(slot), torch.from_numpy(gates).cuda()
        self.q = moe.Fp8Buffers(self.d)
        self.ws = torch.zeros(moe.moe_workspace_size(self.d), dtype=torch.uint8, device="cuda")
        bf = lambda c: torch.full((self.N, c), 7.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.a, self.h, self.o = bf(2 * F), bf(F), bf(H)
        self.d_o, self.da, self.dx = bf(H), bf(2 * F), bf(H)
        self.dgates = torch.zeros(T, k, device="cuda")

    def weights(self):
        q = self.q
        return q.w1q, q.w1s, q.w2q, q.w2s

    def quantize(self):
        self.q.quantize_weights(self.w1, self.w2)

    def permute(self, stream=None):
        moe.moe_permute_fp8(self.d, self.x, self.slot, self.q.xq, self.q.xs, stream)

    def forward(self, save=True, stream=None):
        q = self.q
        moe.moe_expert_ffn_fwd_fp8(self.d, q.xq, q.xs, self.off, *self.weights(),
                                   self.a if save else None, self.h if save else None, q.hq, q.hs,
                                   self.o, self.ws, stream)

    def combine_bwd(self, save=True, stream=None):
        q = self.q
        moe.moe_combine_bwd_fp8(self.d, self.dy, self.o, self.slot, self.gates,
                                self.d_o if save else None, q.dq, q.ds, self.dgates, stream)

    def dgrad(self, save=True, stream=None):
        q = self.q
        moe.moe_expert_ffn_bwd_dgrad_fp8(self.d, q.dq, q.ds, self.a, self.off, *self.weights(),
                                         self.da if save else None, q.daq, q.das, self.dx, self.ws,
                                         stream)

    def status(self):
        assert moe.moe_device_status(self.d, self.ws) == moe.MOE_OK, moe.lib().moe_last_error()

    # oracle views
    def w64(self):
        E, H, F, q = self.E, self.H, self.F, self.q
        w1 = O.values_weights(q64(q.w1q).reshape(2 * E, F, H),
                              q.w1s.cpu().numpy().astype(np.int64).reshape(2 * E, *q.w1s.shape[2:]))
        w2 = O.values_weights(q64(q.w2q), q.w2s.cpu().numpy().astype(np.int64))
        return w1.reshape(E, 2 * F, H), w2

    def rows64(self, q, s, c):
        """(q values, scale bytes) of the first N rows."""
        return q64(q)[: self.N], O.unpack_words(s.cpu().numpy(), -(-c // 128))[: self.N]


CASES = {
    "tiny": dict(T=256, H=128, E=8, k=2, F=256),
    "ragged": dict(T=300, H=192, E=6, k=3, F=192),
    "multi_tile": dict(T=1000, H=320, E=16, k=4, F=448),
    "empty_experts": dict(T=5, H=128, E=16, k=2, F=128, kind="balanced"),
    "dense": dict(T=130, H=128, E=1, k=1, F=128),
    "k_equals_E": dict(T=70, H=64, E=4, k=4, F=64),
    "one_token": dict(T=1, H=2048, E=16, k=8, F=768),
    "one_row": dict(T=1, H=64, E=8, k=1, F=64),
    "wide": dict(T=256, H=1024, E=8, k=2, F=512),
    "large_k": dict(T=150, H=192, E=32, k=20, F=64),
    "max_experts": dict(T=200, H=128, E=256, k=8, F=64),
    "max_hidden": dict(T=40, H=16384, E=2, k=2, F=128),
    "max_inner": dict(T=40, H=128, E=2, k=2, F=16384),
    "one_token_long": dict(T=1, H=4096, E=8, k=2, F=1408),
    "one_token_short": dict(T=1, H=320, E=4, k=4, F=192),
    "one_expert_many_rows": dict(T=40, H=704, E=1, k=1, F=1088),
    "few_rows_odd": dict(T=3, H=704, E=12, k=5, F=320),
    "long_expert": dict(T=700, H=256, E=2, k=2, F=384),
    # few rows an expert on average, a hundred at some: several row tiles
    "few_rows_skewed": dict(T=100, H=320, E=32, k=8, F=448),
    # more than few on average: the 256-row tiles at the largest sizes
    "max_hidden_many_rows": dict(T=64, H=16384, E=1, k=1, F=64),
    "max_inner_many_rows": dict(T=64, H=64, E=1, k=1, F=16384),
    # exactly a tile, one row less and one more
    "tile_256": dict(T=256, H=128, E=1, k=1, F=128),
    "tile_255": dict(T=255, H=128, E=1, k=1, F=192),
    "tile_257": dict(T=257, H=192, E=1, k=1, F=128),
    "tile_129": dict(T=129, H=128, E=1, k=1, F=320),
    # many tiles a CTA pair: every ring and accumulator wraps
    "many_tiles": dict(T=3000, H=512, E=8, k=2, F=576),
    "empty_and_long": dict(T=1500, H=256, E=24, k=1, F=256),
}


@pytest.fixture(scope="module", params=sorted(CASES))
def case(request):
    c = Case(**CASES[request.param], seed=len(request.param))
    c.quantize()
    c.permute()
    c.forward()
    c.combine_bwd()
    c.dgrad()
    c.status()
    return c


def test_weights_bit_exact(case):
    E, H, F, q = case.E, case.H, case.F, case.q
    for name, w, wq, ws in (("w1", np64(case.w1).reshape(2 * E, F, H), q.w1q, q.w1s),
                            ("w2", np64(case.w2), q.w2q, q.w2s)):
        ref, b = O.quantize_weights(w)
        same(name + "q", q64(wq).reshape(ref.shape), ref)
        same(name + "s", ws.cpu().numpy().astype(np.int64).reshape(b.shape), b)


def test_permute_bit_exact(case):
    ref, b = O.quantize_rows(np64(case.x))
    t = np.empty(case.N, np.int64)
    t[case.slot_np.ravel()] = np.arange(case.N) // case.k
    got, gb = case.rows64(case.q.xq, case.q.xs, case.H)
    same("xq", got, ref[t])
    same("xs", gb, b[t])
    nb = b.shape[1]
    pad = np.moveaxis(case.q.xs.cpu().numpy(), 0, 1).reshape(-1, (nb + 3) // 4 * 4)[:, nb:]
    assert (pad == 0).all()


def test_forward_stages(case):
    w1, w2 = case.w64()
    off = case.off_np
    x = O.values_rows(*case.rows64(case.q.xq, case.q.xs, case.H))
    a, h, o = np64(case.a), np64(case.h), np64(case.o)
    r = {"a": close("a", a, O.grouped(x, off, w1),
                    case.H * U32 * O.grouped(np.abs(x), off, np.abs(w1)))}
    ref = O.swiglu(a)
    r["h"] = close("h", h, ref, ELEM * np.abs(ref))
    q, b = O.quantize_rows(h)
    gq, gb = case.rows64(case.q.hq, case.q.hs, case.F)
    same("hq", gq, q)
    same("hs", gb, b)
    hv = O.values_rows(gq, gb)
    r["o"] = close("o", o, O.grouped(hv, off, w2),
                   case.F * U32 * O.grouped(np.abs(hv), off, np.abs(w2)))
    print(r)


def test_combine_bwd_stages(case):
    dy, o, slot = np64(case.dy), np64(case.o), case.slot_np
    g32 = case.gates_np.astype(np.float32)
    prod = (g32[:, :, None] * dy.astype(np.float32)[:, None]).astype(np.float64)  # one fp32 rounding
    d_o = np.empty((case.N, case.H))
    d_o[slot.ravel()] = O.bf16(prod).reshape(-1, case.H)
    same("d_o", np64(case.d_o), d_o)
    q, b = O.quantize_rows(d_o)
    gq, gb = case.rows64(case.q.dq, case.q.ds, case.H)
    same("dq", gq, q)
    same("ds", gb, b)
    pad = np.moveaxis(case.q.ds.cpu().numpy(), 0, 1).reshape(-1, (b.shape[1] + 3) // 4 * 4)[:, b.shape[1]:]
    assert (pad == 0).all()
    terms = dy[:, None] * o[slot]
    err = np.abs(np64(case.dgates) - terms.sum(2))
    assert (err <= case.H * U32 * np.abs(terms).sum(2) + 1e-40).all()


def test_dgrad_stages(case):
    w1, w2 = case.w64()
    off, F = case.off_np, case.F
    d = O.values_rows(*case.rows64(case.q.dq, case.q.ds, case.H))
    a, da, dx = np64(case.a), np64(case.da), np64(case.dx)
    w2t = np.swapaxes(w2, 1, 2)
    dh, acc = O.grouped(d, off, w2t), O.grouped(np.abs(d), off, np.abs(w2t))
    g, u = np.split(a, 2, axis=1)
    s = O.sigmoid(g)
    ref = O.swiglu_grad(dh, a)
    # the gate gradient's factor 1 + g (1 - s) may cancel: its terms' sizes bound its error
    fac = np.concatenate([np.abs(u) * s * (1 + np.abs(g) * (1 - s)), np.abs(g) * s], axis=1)
    dh2, acc2 = np.concatenate([dh, dh], 1), np.concatenate([acc, acc], 1)
    r = {"da": close("da", da, ref, fac * (case.H * U32 * acc2 + ELEM * np.abs(dh2)))}
    q, b = O.quantize_rows(O.halves(da))
    nf = b.shape[1]
    gq = q64(case.q.daq)[: case.N]
    gb = O.unpack_words(case.q.das.cpu().numpy(), 2 * nf)[: case.N]
    same("daq", gq, q.reshape(gq.shape))
    same("das", gb, b.reshape(-1, 2 * nf))
    dv = O.values_rows(q, b).reshape(case.N, 2 * F)
    w1t = np.swapaxes(w1, 1, 2)
    r["dx"] = close("dx_perm", dx, O.grouped(dv, off, w1t),
                    2 * F * U32 * O.grouped(np.abs(dv), off, np.abs(w1t)))
    print(r)


@pytest.mark.parametrize("seed", range(10))
def test_seeded_random_shapes(seed):
    rng = np.random.default_rng(700 + seed)
    E = int(rng.choice([1, 3, 8, 40, 128, 256]))
    c = Case(T=int(rng.choice([1, 2, 17, 64, 200, 900])), H=64 * int(rng.integers(1, 13)), E=E,
             k=int(rng.integers(1, min(E, 8) + 1)), F=64 * int(rng.integers(1, 10)),
             kind=("balanced", "skewed")[seed % 2], seed=seed)
    c.quantize()
    c.permute()
    c.forward()
    c.combine_bwd()
    c.dgrad()
    c.status()
    test_permute_bit_exact(c)
    test_forward_stages(c)
    test_combine_bwd_stages(c)
    test_dgrad_stages(c)


def test_serving_gives_the_same_bits(case):
    """Without a, h, d_o and da the results are those of the calls that store them."""
    o, hq, dq, dx = (t.clone().view(torch.uint8) for t in (case.o, case.q.hq, case.q.dq, case.dx))
    for t in (case.o, case.dx):
        t.fill_(3.0)
    case.q.hq.view(torch.uint8).fill_(0x55)
    case.forward(save=False)
    case.combine_bwd(save=False)
    case.dgrad(save=False)
    case.status()
    for name, got, want in (("o", case.o, o), ("hq", case.q.hq, hq), ("dq", case.q.dq, dq),
                            ("dx", case.dx, dx)):
        assert torch.equal(got.view(torch.uint8), want), name


# ----------------------------------------------------------------------------- values
def special_rows(H):
    """Rows of zeros, of the smallest and the largest bf16 values, with one NaN, one infinity,
    and blocks whose largest magnitude sits at and beside 448 times a power of two."""
    x = torch.randn(12, H, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16)
    x[0] = 0
    x[1] = -0.0
    x[2] = x[2] * 2.0 ** -130  # subnormal in bf16
    x[3] = (x[3].float().clamp(-2, 2) * 2.0 ** 126).to(torch.bfloat16)
    x[4, H // 2] = float("nan")
    x[5, 3] = float("inf")
    x[6, H - 1] = float("-inf")
    x[7] = 2.0 ** -126
    x[8, :64] = 448.0
    x[9, :64] = 450.0  # the next bf16 value
    x[10, :64] = 446.0
    x[11, 0] = 2.0 ** 60  # the others of its block vanish or become subnormal
    return x


@pytest.mark.parametrize("H", [64, 192, 512, 576])
def test_special_values_are_quantised_bit_exact(H):
    x = special_rows(H)
    c = Case(T=12, H=H, E=8, k=2, F=64, x=x, seed=3)
    c.w1.view(-1)[: 12 * H] = x.view(-1).cuda()[: 12 * H]
    c.permute()
    ref, b = O.quantize_rows(np64(x))
    t = np.empty(c.N, np.int64)
    t[c.slot_np.ravel()] = np.arange(c.N) // c.k
    got, gb = c.rows64(c.q.xq, c.q.xs, H)
    same("xq", got, ref[t])
    same("xs", gb, b[t])
    c.quantize()
    wref, wb = O.quantize_weights(np64(c.w1).reshape(16, 64, H))
    same("w1q", q64(c.q.w1q).reshape(wref.shape), wref)
    same("w1s", c.q.w1s.cpu().numpy().astype(np.int64).reshape(wb.shape), wb)
    # gradients of the weighted return
    c.dy.copy_(x)
    c.o.normal_()
    c.combine_bwd()
    d_o = np64(c.d_o)
    q, qb = O.quantize_rows(d_o)
    gq, gqb = c.rows64(c.q.dq, c.q.ds, H)
    same("dq", gq, q)
    same("ds", gqb, qb)


def test_non_finite_rows_stay_in_their_rows():
    x = torch.randn(40, 256, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16)
    clean = Case(T=40, H=256, E=4, k=2, F=192, x=x, seed=6)
    bad_x = x.clone()
    bad_x[7, 100], bad_x[31, 0] = float("nan"), float("inf")
    bad = Case(T=40, H=256, E=4, k=2, F=192, x=bad_x, seed=6)
    for c in (clean, bad):
        c.quantize()
        c.permute()
        c.forward()
        c.status()
    rows = np.zeros(80, bool)
    rows[clean.slot_np[[7, 31]].ravel()] = True
    o, want = np64(bad.o), np64(clean.o)
    assert np.isnan(o[rows]).all()
    same("o", o[~rows], want[~rows])
    # and the same for the gradient
    for c, dy in ((clean, x), (bad, bad_x)):
        c.dy.copy_(dy)
        c.a.copy_(clean.a)
        c.o.copy_(clean.o)
        c.combine_bwd()
        c.dgrad()
    dx, dwant = np64(bad.dx), np64(clean.dx)
    assert np.isnan(dx[rows]).all()
    same("dx", dx[~rows], dwant[~rows])


def test_a_non_finite_weight_stays_in_its_expert():
    c = Case(T=60, H=192, E=4, k=2, F=192, seed=7)
    c.quantize()
    c.permute()
    c.forward()
    c.combine_bwd()
    c.dgrad()
    o, dx = np64(c.o), np64(c.dx)
    lo, hi = int(c.off_np[1]), int(c.off_np[2])
    mine = np.zeros(c.N, bool)
    mine[lo:hi] = True
    assert mine.any() and not mine.all()
    # last rows and columns: they share TMA boxes with the next expert's
    c.w1[1, -1, -1] = float("nan")
    c.w2[1, -1, -1] = float("inf")
    c.quantize()
    c.forward()
    c.a[:] = 0.5  # (the forward's own a of that expert is NaN)
    c.dgrad()
    c.status()
    same("o", np64(c.o)[~mine], o[~mine])
    assert np.isnan(np64(c.o)[mine]).any() and np.isnan(np64(c.dx)[mine]).any()
    assert np.isfinite(np64(c.dx)[~mine]).all()


@pytest.mark.parametrize("power", [-60, 40])
def test_power_of_two_scaling_is_exact(power):
    """x 2^p gives a 2^p bit for bit: the scales carry it, the sums see the same e4m3 values."""
    x = torch.randn(50, 320, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16)
    c1 = Case(T=50, H=320, E=4, k=2, F=64, x=x, seed=8)
    c2 = Case(T=50, H=320, E=4, k=2, F=64, x=(x.float() * 2.0 ** power).to(torch.bfloat16), seed=8)
    for c in (c1, c2):
        c.quantize()
        c.permute()
        c.forward()
    same("a", np64(c2.a), np64(c1.a) * 2.0 ** power)


# ----------------------------------------------------------------------------- rows and slots
def test_rows_behind_the_last_and_skipped_slots_are_left_alone():
    c = Case(T=50, H=192, E=4, k=2, F=192, seed=10)
    c.quantize()
    u8 = lambda t: t.view(torch.uint8)  # noqa: E731
    u8(c.q.xq).fill_(0x2A)
    c.q.xs.fill_(77)
    c.slot[3, 1] = -1
    c.slot[4, 0] = c.N  # one past the last row
    c.permute()
    for s in (c.slot_np[3, 1], c.slot_np[4, 0]):
        assert (u8(c.q.xq)[s] == 0x2A).all() and (c.q.xs[:, s] == 77).all()
    u8(c.q.dq).fill_(0x2A)
    c.o.normal_()
    c.d_o.fill_(7.0)
    c.combine_bwd()
    for s in (c.slot_np[3, 1], c.slot_np[4, 0]):
        assert (u8(c.q.dq)[s] == 0x2A).all() and (c.d_o[s] == 7).all()
    assert float(c.dgates[3, 1]) == 0 and float(c.dgates[4, 0]) == 0
    # fewer rows than N: those past off[E] keep what they held; offsets past N are bounds
    for last, off in ((c.N - 9, None), (c.N, c.N + 1000)):
        c.slot.copy_(torch.from_numpy(c.slot_np.astype(np.int32)))
        c.permute()
        c.off.copy_(torch.from_numpy(np.minimum(c.off_np, last).astype(np.int32)))
        if off:
            c.off[-1] = off
        for t in (c.a, c.h, c.o, c.da, c.dx):
            t.fill_(7.0)
        u8(c.q.hq).fill_(0x2A)
        c.forward()
        a = c.a.clone()
        c.a.normal_()
        c.dgrad()
        c.status()
        for t in (a, c.h, c.o, c.da, c.dx):
            assert (t[last:] == 7).all() and not (t[:last] == 7).all(1).any()
        assert (u8(c.q.hq)[last:] == 0x2A).all()


def test_offsets_out_of_order_write_nothing_outside():
    c = Case(T=50, H=128, E=4, k=2, F=128, seed=11)
    c.quantize()
    c.permute()
    c.off.copy_(torch.tensor([-5, 60, 20, 1 << 30, 100], dtype=torch.int32))
    guard = torch.full((c.N + 256, c.H), 7.0, dtype=torch.bfloat16, device="cuda")
    c.o = guard[128:128 + c.N]
    c.forward()
    c.status()
    assert (guard[:128] == 7).all() and (guard[128 + c.N:] == 7).all()


@pytest.mark.parametrize("T", [0])
def test_no_tokens(T):
    d = moe.LayerDesc.of(T, 128, 8, 2, 128)
    b, q = moe.LayerBuffers(d), moe.Fp8Buffers(d)
    q.quantize_weights(b.w1, b.w2)
    moe.moe_layer_forward_fp8(d, b, q)
    b.dw1.fill_(3.0)
    moe.moe_layer_backward_fp8(d, b, q)
    assert moe.moe_device_status(d, b.ws) == moe.MOE_OK
    assert float(b.dw1.abs().max()) == 0


def test_no_tokens_without_the_saved_buffers():
    c = Case(T=1, H=192, E=4, k=2, F=128, seed=25)
    c.d = moe.LayerDesc.of(0, 192, 4, 2, 128)
    c.off.zero_()
    c.forward(save=False)
    c.combine_bwd(save=False)
    c.dgrad(save=False)
    c.status()
    assert float(c.o.min()) == 7 and float(c.dx.min()) == 7


# ----------------------------------------------------------------------------- streams, graphs
def test_side_stream_and_repeat_give_the_same_bits():
    c = Case(T=300, H=320, E=8, k=4, F=192, seed=12)
    st = torch.cuda.Stream()
    outs = []
    for stream in (None, st, st):
        for t in (c.a, c.h, c.o, c.d_o, c.da, c.dx):
            t.zero_()
        torch.cuda.synchronize()
        c.quantize()
        torch.cuda.synchronize()
        c.permute(stream)
        c.forward(stream=stream)
        c.combine_bwd(stream=stream)
        c.dgrad(stream=stream)
        torch.cuda.synchronize()
        outs.append([t.clone() for t in (c.a, c.h, c.o, c.d_o, c.dgates, c.da, c.dx)])
    for later in outs[1:]:
        for x, y in zip(outs[0], later):
            assert torch.equal(x, y)


def test_two_calls_at_once_with_workspaces_of_their_own():
    cs = [Case(T=400, H=256, E=8, k=4, F=256, seed=s) for s in (13, 14)]
    want = []
    for c in cs:
        c.quantize()
        c.permute()
        c.forward()
        want.append(c.o.clone())
        c.o.zero_()
    torch.cuda.synchronize()
    sts = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for c, st in zip(cs, sts):
            c.forward(stream=st)
    torch.cuda.synchronize()
    for c, w in zip(cs, want):
        c.status()
        assert torch.equal(c.o, w)


def test_chains_of_every_kind_at_once():
    # forwards of many and of few rows and a gradient, each with more tiles than CTAs
    # or sharing the SMs with one that has: none may wait for a CTA that is not there
    many, few, grad = (Case(T=T, H=512, E=32, k=4, F=512, seed=s)
                       for T, s in ((2500, 21), (200, 22), (2500, 23)))
    want = []
    for c in (many, few, grad):
        c.quantize()
        c.permute()
        c.forward()
        c.combine_bwd()
        c.dgrad()
        want.append([t.clone() for t in (c.o, c.da, c.dx)])
        c.o.zero_()
        c.dx.zero_()
    torch.cuda.synchronize()
    sts = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(8):
        many.forward(stream=sts[0])
        few.forward(stream=sts[1])
        grad.dgrad(stream=sts[2])
        few.forward(stream=sts[1])
    torch.cuda.synchronize()
    for c in (many, few, grad):
        c.status()
    assert torch.equal(many.o, want[0][0]) and torch.equal(few.o, want[1][0])
    assert torch.equal(grad.da, want[2][1]) and torch.equal(grad.dx, want[2][2])


@pytest.mark.parametrize("H", [64, 512])
def test_short_products_with_long_epilogues_repeat(H):
    # the gradient's first product is over long before its epilogue: the second one's
    # operands may not take the pre-activations' memory yet
    c = Case(T=6000, H=H, E=8, k=2, F=576, seed=24)
    c.quantize()
    c.permute()
    c.forward()
    c.combine_bwd()
    want = None
    for _ in range(20):
        c.da.zero_()
        c.dx.zero_()
        c.dgrad()
        got = (c.da.clone(), c.q.daq.view(torch.uint8).clone(), c.dx.clone())
        want = want or got
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    c.status()
    test_dgrad_stages(c)


@pytest.mark.parametrize("T", [1, 200])
def test_captured_and_replayed(T):
    c = Case(T=T, H=256, E=8, k=4, F=192, seed=15)
    c.quantize()

    def run():
        c.permute()
        c.forward()
        c.combine_bwd()
        c.dgrad()

    run()  # first calls set kernel attributes up
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for seed in (1, 2):
        gen = torch.Generator().manual_seed(seed)
        c.x.copy_(torch.randn(T, 256, generator=gen))
        c.dy.copy_(torch.randn(T, 256, generator=gen))
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (c.o, c.dgates, c.dx)]
        run()
        torch.cuda.synchronize()
        for x, y in zip(got, (c.o, c.dgates, c.dx)):
            assert torch.equal(x, y)


@pytest.mark.parametrize("wgrad", [True, False])
def test_layer_captured_and_replayed(wgrad):
    """Forward and backward of the layer (the side stream's fork and join inside) in one graph."""
    inp = moe_synth.make_inputs(T=200, H=128, E=8, k=2, F=192, seed=38)
    d = moe.LayerDesc.of(**inp.shape_dict())
    b, q = moe.LayerBuffers(d), moe.Fp8Buffers(d)
    b.load_inputs(inp)
    q.quantize_weights(b.w1, b.w2)

    def run():
        moe.moe_layer_forward_fp8(d, b, q)
        moe.moe_layer_backward_fp8(d, b, q, run_wgrad=wgrad)

    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    other = moe_synth.make_inputs(T=200, H=128, E=8, k=2, F=192, seed=39)
    b.x.copy_(other.x)
    b.dy.copy_(other.dy)
    g.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (b.y, b.dx, b.dw_r, b.dw1, b.dw2)]
    run()
    torch.cuda.synchronize()
    assert moe.moe_device_status(d, b.ws) == moe.MOE_OK
    for x, y in zip(got, (b.y, b.dx, b.dw_r, b.dw1, b.dw2)):
        assert torch.equal(x, y)


# ----------------------------------------------------------------------------- offsets past 32 bits
def test_buffers_past_32_bits():
    """Rows whose element offsets pass 2^31 in every buffer: the last rows against the oracle."""
    T, H, E, k, F = 75000, 4096, 8, 8, 64
    N = T * k
    assert N * H > 2 ** 31
    d = moe.LayerDesc.of(T, H, E, k, F)
    g = torch.Generator(device="cuda").manual_seed(40)
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(torch.bfloat16)  # noqa: E731
    q = moe.Fp8Buffers(d)
    q.quantize_weights(rnd(E, 2 * F, H, std=0.02), rnd(E, H, F, std=0.05))
    x = rnd(T, H)
    # every token to every expert: row s of expert e is token s - e T
    off = (torch.arange(E + 1, device="cuda") * T).to(torch.int32)
    slot = (torch.arange(T, device="cuda")[:, None] + T * torch.arange(E, device="cuda")).to(torch.int32)
    gates = torch.full((T, k), 0.125, device="cuda")
    new = lambda c: torch.zeros(N, c, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    a, h, o, d_o, dx = new(2 * F), new(F), new(H), new(H), new(H)
    dgates = torch.zeros(T, k, device="cuda")
    ws = torch.zeros(moe.moe_workspace_size(d), dtype=torch.uint8, device="cuda")
    w = (q.w1q, q.w1s, q.w2q, q.w2s)
    moe.moe_permute_fp8(d, x, slot, q.xq, q.xs)
    moe.moe_expert_ffn_fwd_fp8(d, q.xq, q.xs, off, *w, a, h, q.hq, q.hs, o, ws)
    moe.moe_combine_bwd_fp8(d, x, o, slot, gates, d_o, q.dq, q.ds, dgates)
    moe.moe_expert_ffn_bwd_dgrad_fp8(d, q.dq, q.ds, a, off, *w, None, q.daq, q.das, dx, ws)
    assert moe.moe_device_status(d, ws) == moe.MOE_OK
    rows = np.r_[N - 40:N]  # of the last expert
    w1 = O.values_weights(q64(q.w1q[-1]).reshape(2, F, H), q.w1s[-1].cpu().numpy().astype(np.int64)).reshape(1, 2 * F, H)
    w2 = O.values_weights(q64(q.w2q[-1:]), q.w2s[-1:].cpu().numpy().astype(np.int64))
    one = np.array([0, len(rows)])
    tail = lambda t: np64(t[N - 40:])  # noqa: E731
    scales = lambda s, nb: O.unpack_words(s[:, N - 40:].cpu().numpy(), nb)  # noqa: E731
    ref, b = O.quantize_rows(np64(x[T - 40:]))
    same("xq", q64(q.xq[N - 40:]), ref)
    same("xs", scales(q.xs, H // 128), b)
    xv = O.values_rows(ref, b)
    close("a", tail(a), O.grouped(xv, one, w1), H * U32 * O.grouped(np.abs(xv), one, np.abs(w1)))
    hq, hb = O.quantize_rows(tail(h))
    same("hq", q64(q.hq[N - 40:]), hq)
    hv = O.values_rows(hq, hb)
    close("o", tail(o), O.grouped(hv, one, w2), F * U32 * O.grouped(np.abs(hv), one, np.abs(w2)))
    same("d_o", tail(d_o), O.bf16(0.125 * np64(x[T - 40:])))
    dq, db = O.quantize_rows(tail(d_o))
    same("dq", q64(q.dq[N - 40:]), dq)
    same("ds", scales(q.ds, H // 128), db)
    dv = O.values_rows(q64(q.daq[N - 40:]).reshape(80, F), scales(q.das, 2).reshape(80, 1)).reshape(40, 2 * F)
    w1t = np.swapaxes(w1, 1, 2)
    close("dx", tail(dx), O.grouped(dv, one, w1t), 2 * F * U32 * O.grouped(np.abs(dv), one, np.abs(w1t)))


# ----------------------------------------------------------------------------- the whole layer
LAYERS = {
    "tiny": dict(T=256, H=128, E=8, k=2, F=256, seed=31),
    "ragged": dict(T=300, H=192, E=6, k=3, F=192, seed=32),
    "more_than_128_experts": dict(T=90, H=128, E=256, k=4, F=64, seed=33),
    "skewed": dict(T=500, H=256, E=32, k=8, F=320, seed=34, bias="zipf_logrank"),
    "one_token": dict(T=1, H=256, E=8, k=2, F=128, seed=35),
}


@pytest.mark.parametrize("name", sorted(LAYERS))
def test_layer_is_its_calls_in_order(name):
    """The layer calls against the entry points one by one, bit for bit, and against
    the bf16 layer in what they share."""
    inp = moe_synth.make_inputs(**LAYERS[name])
    d = moe.LayerDesc.of(**inp.shape_dict())
    b, q = moe.LayerBuffers(d), moe.Fp8Buffers(d)
    b.load_inputs(inp)
    q.quantize_weights(b.w1, b.w2)
    moe.moe_layer_forward_fp8(d, b, q)
    moe.moe_layer_backward_fp8(d, b, q)
    assert moe.moe_device_status(d, b.ws) == moe.MOE_OK
    r, rq = moe.LayerBuffers(d), moe.Fp8Buffers(d, weights=q)
    r.load_inputs(inp)
    moe.moe_dispatch_fused(d, r.x, r.w_r, r.bias, r.logits, r.idx, r.gates, r.cnt, r.off, r.slot,
                           r.row_src, r.cnt_re, r.rank_off, r.x_perm, r.ws)
    w = (q.w1q, q.w1s, q.w2q, q.w2s)
    moe.moe_permute_fp8(d, r.x, r.slot, rq.xq, rq.xs)
    moe.moe_expert_ffn_fwd_fp8(d, rq.xq, rq.xs, r.off, *w, r.a, r.h, rq.hq, rq.hs, r.o, r.ws)
    moe.moe_combine(d, r.o, r.slot, r.gates, r.y)
    moe.moe_combine_bwd_fp8(d, r.dy, r.o, r.slot, r.gates, r.d_o, rq.dq, rq.ds, r.dgates)
    moe.moe_expert_ffn_bwd_dgrad_fp8(d, rq.dq, rq.ds, r.a, r.off, *w, r.da, rq.daq, rq.das,
                                     r.dx_perm, r.ws)
    moe.moe_permute_bwd(d, r.dx_perm, r.slot, r.dx32)
    moe.moe_route_bwd(d, r.dgates, r.gates, r.idx, r.x, r.w_r, r.row_src, r.off, r.dx32, r.dx,
                      r.dw_r, r.ws)
    moe.moe_expert_ffn_bwd_wgrad(d, r.x_perm, r.h, r.d_o, r.da, r.off, r.dw1, r.dw2, r.ws)
    torch.cuda.synchronize()
    for n in ("idx", "slot", "off", "gates", "x_perm", "a", "h", "o", "y", "d_o", "dgates", "da",
              "dx_perm", "dx", "dw_r", "dw1", "dw2"):
        assert torch.equal(getattr(b, n), getattr(r, n)), n
    # serving: the same y without x_perm, a and h
    s, sq = moe.LayerBuffers(d, weights=b), moe.Fp8Buffers(d, weights=q, backward=False)
    s.x.copy_(b.x)
    s.x_perm = s.a = s.h = None
    moe.moe_layer_forward_fp8(d, s, sq, save=False)
    assert moe.moe_device_status(d, s.ws) == moe.MOE_OK
    assert torch.equal(s.y, b.y)
    # frozen experts: the same dx without the weight gradients and their inputs
    dx = b.dx.clone()
    b.d_o = b.da = None
    b._struct = None
    moe.moe_layer_backward_fp8(d, b, q, run_wgrad=False)
    torch.cuda.synchronize()
    assert torch.equal(b.dx, dx)


def test_layer_is_near_the_bf16_layer():
    """An e4m3 value is off by at most 2^-4 of itself, so each of the two rounded factors of a
    product adds at most 2^-4 (1 + 2^-4): the sums' errors stay under 2^-4 * 2.1 of the sum of the
    magnitudes of their terms, for o with h's own error on top. As that bound is wide and the
    errors are independent of sign, the norm of y's difference stays far inside it: half of it."""
    inp = moe_synth.make_inputs(T=512, H=256, E=8, k=2, F=256, seed=36)
    d = moe.LayerDesc.of(**inp.shape_dict())
    b, r, q = moe.LayerBuffers(d), moe.LayerBuffers(d), moe.Fp8Buffers(d)
    for t in (b, r):
        t.load_inputs(inp)
    q.quantize_weights(b.w1, b.w2)
    moe.moe_layer_forward_fp8(d, b, q)
    moe.moe_layer_backward_fp8(d, b, q)
    moe.moe_layer_forward(d, r)
    moe.moe_layer_backward(d, r)
    for n in ("y", "dw1", "dw2", "dx_perm"):
        x, y = getattr(b, n).float(), getattr(r, n).float()
        rel = float((x - y).norm() / y.norm())
        print(n, rel)
        assert 0 < rel < 2.1 * 2.0 ** -4


def test_accumulating_weight_gradients():
    inp = moe_synth.make_inputs(T=128, H=128, E=4, k=2, F=128, seed=37)
    d0 = moe.LayerDesc.of(**inp.shape_dict())
    d1 = moe.LayerDesc.of(**inp.shape_dict(), flags=moe.FLAG_WGRAD_ACCUM_FP32)
    b0, b1, q = moe.LayerBuffers(d0), moe.LayerBuffers(d1), moe.Fp8Buffers(d0)
    for d, b in ((d0, b0), (d1, b1)):
        b.load_inputs(inp)
        q.quantize_weights(b.w1, b.w2)
        moe.moe_layer_forward_fp8(d, b, q)
        moe.moe_layer_backward_fp8(d, b, q)
    assert torch.equal(b1.main_dw1.to(torch.bfloat16), b0.dw1)
    assert torch.equal(b1.main_dw2.to(torch.bfloat16), b0.dw2)
