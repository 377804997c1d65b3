"""The input norm of finite rows whose squares leave fp32's range, against the float64 oracle.

Bounds. Such a row is summed under a power of two, so its sum errs as any other row's:
(H + 1) 2^-24 of itself, rstd by half of that and a few roundings: (H / 2 + 8) 2^-24. rstd
itself may be below fp32's normal range, but is 2^-128 at least (a bf16 is below 2^128): half a
step of 2^-149 is 2^-22 of that. y: two products and a bf16 rounding more, and half of bf16's
smallest step, 2^-134."""
import numpy as np
import pytest
import torch

import combine_router_softmax_top_gb300 as moe
from oracle import fp4_oracle as Q

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
BIG, TINY = float(torch.finfo(BF).max), 2.0 ** -133


@pytest.fixture(scope="module", autouse=True)
def built():
    from combine_router_softmax_top_gb300 import build
    build.build()


def f64(t):
    return t.detach().double().cpu().numpy()


def desc(T, H):
    return moe.LayerDesc.of(T, H, 1, 1, 64)


def norm(x, res, w, eps):
    T, H = x.shape
    r = torch.empty_like(x) if res is not None else None
    y, rstd = torch.empty_like(x), torch.empty(T, device="cuda")
    yq = torch.zeros(T, H, device="cuda").to(torch.float8_e4m3fn)
    ys = torch.zeros(-(-H // 512), T, 4, dtype=torch.uint8, device="cuda")
    moe.moe_rms_norm(desc(T, H), x, res, w, eps, r, y, yq, ys, rstd)
    return (x if r is None else r), y, rstd, yq, ys


def check(r, y, rstd, w, eps, rows):
    H = r.shape[1]
    want, want_rstd = Q.rms_norm(f64(r)[rows], f64(w), eps)
    rel = (H / 2 + 8) * 2.0 ** -24 + 2.0 ** -22
    assert (np.abs(f64(rstd)[rows] - want_rstd) <= rel * want_rstd).all()
    assert (np.abs(f64(y)[rows] - want) <= (rel + 2.0 ** -8 + 2.0 ** -22) * np.abs(want) + 2.0 ** -134).all()


# every way a row is dealt to threads: parts of a warp, one, two rows a block, one row a block;
# the last two with four groups of columns a thread
SHAPES = [(7, 64), (9, 128), (5, 320), (9, 512), (7, 704), (6, 1024), (5, 2048), (3, 16384),
          (400, 1024), (160, 4096), (160, 16384)]


def rows_of(T, H, scales, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, H, generator=g, device="cuda").clamp(-4, 4)
    s = torch.tensor([scales[i % len(scales)] for i in range(T)], device="cuda", dtype=torch.float64)
    return (x.double() * s[:, None]).clamp(-BIG, BIG).to(BF)


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("residual", [True, False])
def test_large_rows(T, H, residual):
    """Rows of 1e20 to the largest bf16, among ordinary ones, whose bits they leave alone."""
    scales = [1.0, 1e20, 2.0 ** 126, 3.0, 1e19, 2.0 ** 64]
    x = rows_of(T, H, scales)
    res = rows_of(T, H, [0.5], seed=1) if residual else None
    w = (1 + 0.2 * rows_of(1, H, [1.0], seed=2)[0].float()).to(BF)
    r, y, rstd, yq, ys = norm(x, res, w, 1e-6)
    assert torch.isfinite(r.float()).all()
    check(r, y, rstd, w, 1e-6, slice(None))
    assert (y.float().abs().amax(1) > 0.5).all()
    small = torch.tensor([scales[i % len(scales)] < 10 for i in range(T)], device="cuda")
    x2, res2 = x.clone(), None if res is None else res.clone()
    x2[~small] = 1
    _, y2, rstd2, yq2, _ = norm(x2, res2, w, 1e-6)
    assert torch.equal(y[small], y2[small]) and torch.equal(rstd[small], rstd2[small])
    assert torch.equal(yq.view(torch.uint8)[small], yq2.view(torch.uint8)[small])


@pytest.mark.parametrize("T,H", SHAPES)
def test_tiny_rows_without_eps(T, H):
    """eps = 0: rows down to the smallest normal bf16, some 2^-126; a row of zeros is 0 / 0."""
    scales = [2.0 ** -70, 1.0, 2.0 ** -90, 2.0 ** -122, 0.0]
    x = rows_of(T, H, scales)
    w = torch.ones(H, dtype=BF, device="cuda")
    r, y, rstd, _, _ = norm(x, None, w, 0.0)
    zero = np.array([scales[i % len(scales)] == 0 for i in range(T)])
    check(r, y, rstd, w, 0.0, ~zero)
    assert torch.isnan(y[torch.tensor(zero, device="cuda")].float()).all()


def test_one_large_element():
    """The others of its row are 0 or next to it, as the definition has them."""
    T, H = 4, 2048
    x = torch.ones(T, H, device="cuda").to(BF)
    for t, (c, v) in enumerate([(0, 1e30), (777, -1e25), (2047, BIG), (5, 2.0 ** 63)]):
        x[t, c] = v
    w = torch.full((H,), 2.0, dtype=BF, device="cuda")
    r, y, rstd, _, _ = norm(x, None, w, 1e-5)
    check(r, y, rstd, w, 1e-5, slice(None))


@pytest.mark.parametrize("eps", [1e-6, 2.0 ** -95, 2.0 ** -110, 1e38, 3.4e38])
def test_eps_decides_beside_small_or_large_rows(eps):
    T, H = 6, 320
    x = rows_of(T, H, [2.0 ** -60, 2.0 ** -45, 2.0 ** -120, 0.0, 1.0, 1e19], seed=3)
    w = torch.ones(H, dtype=BF, device="cuda")
    r, y, rstd, _, _ = norm(x, None, w, eps)
    check(r, y, rstd, w, float(np.float32(eps)), slice(None))


def test_what_is_not_finite_stays_so():
    """A NaN makes its whole row NaN; an infinity is NaN itself and the rest of its row 0, also
    beside large elements."""
    T, H = 6, 1024
    x = rows_of(T, H, [1e20])
    x[1, 3], x[2, 900], x[4, 0], x[4, 1] = float("nan"), float("inf"), float("-inf"), float("nan")
    w = torch.ones(H, dtype=BF, device="cuda")
    r, y, rstd, _, _ = norm(x, None, w, 1e-6)
    check(r, y, rstd, w, 1e-6, [0, 3, 5])
    nan = torch.isnan(y.float())
    assert nan[1].all() and nan[4].all()
    assert nan[2, 900] and nan[2].sum() == 1 and (y[2, :900].float() == 0).all() and rstd[2] == 0


@pytest.mark.parametrize("T,H", [(9, 320), (6, 2048)])
def test_gradient_of_large_rows(T, H):
    """With the forward's rstd. xh is of order one, so dx is as small as rstd; dw takes part of
    every row. Bounds as in the norm's other tests, rstd's bits aside (it is the input here)."""
    x = rows_of(T, H, [1e20, 1.0, 2.0 ** 100])
    w = (1 + 0.2 * rows_of(1, H, [1.0], seed=2)[0].float()).to(BF)
    dy = rows_of(T, H, [1.0], seed=4)
    r, _, rstd, _, _ = norm(x, None, w, 1e-6)
    dx, dw = torch.empty_like(x), torch.empty(H, device="cuda")
    d = desc(T, H)
    ws = torch.empty(moe.moe_rms_norm_bwd_workspace_size(d), dtype=torch.uint8, device="cuda")
    moe.moe_rms_norm_bwd(d, dy, None, r, w, rstd, dx, dw, ws)
    want, want_dw = Q.rms_norm_bwd(f64(dy), f64(r), f64(w), f64(rstd))
    xh, g = f64(r) * f64(rstd)[:, None], f64(dy) * f64(w)
    dot = np.abs(g * xh).sum(1, keepdims=True) / H
    err = f64(rstd)[:, None] * ((H + 3) * 2.0 ** -24 * dot * np.abs(xh)
                                + 8 * 2.0 ** -24 * (np.abs(g) + np.abs(xh) * dot))
    assert (np.abs(f64(dx) - want) <= err + 2.0 ** -8 * np.abs(want) + 2.0 ** -134).all()
    assert (np.abs(f64(dw) - want_dw) <= (T + 4) * 2.0 ** -24 * np.abs(f64(dy) * xh).sum(0)).all()
