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


# 4 experts, 2 a token: 25 rows an expert for the few-rows kernel, 200 for the chain, whose tiles
# then have whole boxes of 32 rows, a ragged last one, and rows for both CTAs of a pair at some
BOTH = pytest.mark.parametrize("T,kernel", [(50, "fp8_rows_ffn"), (400, "fp8_gemm_ffn_fwd")])


def forward(c, kernel, **kw):
    assert kernel in kernels(lambda: c.forward(**kw))


@BOTH
@pytest.mark.parametrize("save", [True, False])
def test_non_finite_rows_stay_in_their_rows(T, kernel, save):
    x = torch.randn(T, 256, generator=torch.Generator().manual_seed(51)).to(torch.bfloat16)
    bad_x = x.clone()
    tokens = [7, 31, T - 1]
    bad_x[7, 100], bad_x[31, 0], bad_x[T - 1, 255] = float("nan"), float("inf"), float("-inf")
    clean, bad = (G.Case(T=T, H=256, E=4, k=2, F=192, x=v, seed=52) for v in (x, bad_x))
    for c in (clean, bad):
        c.quantize()
        c.permute()
        forward(c, kernel, save=save)
        c.status()
    rows = np.zeros(2 * T, bool)
    rows[clean.slot_np[tokens].ravel()] = True
    assert np.isfinite(G.np64(clean.o)).all()
    for n in ("a", "h", "o") if save else ("o",):
        got, want = G.np64(getattr(bad, n)), G.np64(getattr(clean, n))
        assert np.isnan(got[rows]).all(), n
        G.same(n, got[~rows], want[~rows])
    clean.forward()  # (a is the gradient's input)
    for c, dy in ((clean, x), (bad, bad_x)):
        c.dy.copy_(dy)
        c.a.copy_(clean.a)
        c.o.copy_(clean.o)
        c.combine_bwd(save=save)
        c.dgrad(save=save)
        c.status()
    for n in ("da", "dx") if save else ("dx",):
        got, want = G.np64(getattr(bad, n)), G.np64(getattr(clean, n))
        assert np.isnan(got[rows]).all(), n
        G.same(n, got[~rows], want[~rows])


@BOTH
def test_a_non_finite_weight_stays_in_its_expert(T, kernel):
    c = G.Case(T=T, H=192, E=4, k=2, F=192, seed=53)
    c.quantize()
    c.permute()
    forward(c, kernel)
    c.combine_bwd()
    c.a[:] = 0.5
    c.dgrad()
    o, dx = G.np64(c.o), G.np64(c.dx)
    lo, hi = int(c.off_np[1]), int(c.off_np[2])
    mine = np.zeros(c.N, bool)
    mine[lo:hi] = True
    assert mine.any() and not mine.all()
    # last rows and columns: they share TMA boxes with the next expert's
    c.w1[1, -1, -1] = float("nan")
    c.w2[1, -1, -1] = float("inf")
    c.quantize()
    forward(c, kernel)
    c.a[:] = 0.5  # (the forward's own a of that expert is NaN)
    c.dgrad()
    c.status()
    for name, got, want in (("o", c.o, o), ("dx", c.dx, dx)):
        got = G.np64(got)
        G.same(name, got[~mine], want[~mine])
        # a NaN in one block of a weight reaches every row of its expert
        assert np.isnan(got[mine]).any(1).all(), name


@BOTH
@pytest.mark.parametrize("power", [-60, 40])
def test_power_of_two_scaling_is_exact(T, kernel, power):
    """x 2^p gives a 2^p bit for bit: the scales carry it, the sums see the same e4m3 values."""
    x = torch.randn(T, 320, generator=torch.Generator().manual_seed(54)).to(torch.bfloat16)
    c1 = G.Case(T=T, H=320, E=4, k=2, F=64, x=x, seed=54)
    c2 = G.Case(T=T, H=320, E=4, k=2, F=64, x=(x.float() * 2.0 ** power).to(torch.bfloat16), seed=54)
    for c in (c1, c2):
        c.quantize()
        c.permute()
        forward(c, kernel)
        c.status()
    G.same("a", G.np64(c2.a), G.np64(c1.a) * 2.0 ** power)


@BOTH
@pytest.mark.parametrize("short", [0, 9, 45])
def test_rows_behind_the_last_are_left_alone(T, kernel, short):
    """off[E] < N (and, with short = 0, offsets past N, which are bounds): the rows that no expert
    has keep what they held, the others are those of the oracle."""
    c = G.Case(T=T, H=192, E=4, k=2, F=192, seed=55)
    c.quantize()
    c.permute()
    last = c.N - short
    c.off_np = np.minimum(c.off_np, last)
    c.off.copy_(torch.from_numpy(c.off_np.astype(np.int32)))
    if not short:
        c.off[-1] = c.N + 1000
    u8 = lambda t: t.view(torch.uint8)  # noqa: E731
    for t in (c.a, c.h, c.o, c.da, c.dx):
        t.fill_(7.0)
    for t in (c.q.hq, c.q.daq):
        u8(t).fill_(0x2A)
    for t in (c.q.hs, c.q.das):
        t.fill_(77)
    forward(c, kernel)
    c.combine_bwd()
    a = c.a.clone()
    c.a[last:].normal_()  # rows that the gradient may not read
    c.dgrad()
    c.status()
    for t in (a, c.h, c.o, c.da, c.dx):
        assert (t[last:] == 7).all() and not (t[:last] == 7).all(1).any()
    for t in (c.q.hq, c.q.daq):
        assert (u8(t)[last:] == 0x2A).all()
    for t in (c.q.hs, c.q.das):
        assert (t[:, last:] == 77).all()
    cut = G.Case.__new__(G.Case)
    cut.__dict__.update(c.__dict__)
    cut.N = last
    for n in ("h", "o", "da", "dx"):
        setattr(cut, n, getattr(c, n)[:last])
    cut.a = a[:last]
    G.test_forward_stages(cut)
    G.test_dgrad_stages(cut)


@BOTH
@pytest.mark.parametrize("save", [True, False])
def test_offsets_out_of_order_write_nothing_outside(T, kernel, save):
    """Every output of the forward and of the gradient between guard rows."""
    c = G.Case(T=T, H=128, E=4, k=2, F=192, seed=56)
    c.quantize()
    c.permute()
    c.combine_bwd()
    N, pad = c.N, 160
    assert N >= 100
    c.off.copy_(torch.tensor([-5, N // 2 + 10, 20, 1 << 30, 100], dtype=torch.int32))
    guards = []

    def guarded(shape, dtype):
        n = int(np.prod(shape))
        row = pad * shape[-1] if len(shape) == 2 else 4096
        size = torch.empty(0, dtype=dtype).element_size()
        raw = torch.full(((n + 2 * row) * size,), 0x2A, dtype=torch.uint8, device="cuda")
        guards.append((raw, row * size))
        return raw[row * size: (row + n) * size].view(dtype).view(*shape)

    bf, e4, u8 = torch.bfloat16, torch.float8_e4m3fn, torch.uint8
    c.a, c.h, c.o = (guarded((N, w), bf) for w in (384, 192, 128))
    c.da, c.dx = guarded((N, 384), bf), guarded((N, 128), bf)
    c.q.hq, c.q.daq = guarded((N, 192), e4), guarded((N, 384), e4)
    c.q.hs, c.q.das = guarded((1, N, 4), u8), guarded((1, N, 4), u8)
    forward(c, kernel, save=save)
    c.a.fill_(0.5)
    c.dgrad(save=save)
    c.status()
    for raw, g in guards:
        assert (raw[:g] == 0x2A).all() and (raw[-g:] == 0x2A).all()
    assert not (c.o.view(u8) == 0x2A).all() and not (c.dx.view(u8) == 0x2A).all()
