"""The layer's input norm and its gradient on the GPU against the float64 oracle.

Bounds. r is one fp32 addition rounded to bf16: half a step of the exact sum, and one fp32
rounding. rstd: the fp32 sum of H squares, each rounded, in any order, errs by (H + 1) 2^-24
of itself at most, so rstd by half of that and a few roundings: (H / 2 + 8) 2^-24. y: that, two
products and a bf16 rounding. dx: its dot product errs by (H + 3) 2^-24 sum |g xh|; dw by
(T + 2) 2^-24 sum |dy xh|."""
import numpy as np
import pytest
import torch

import combine_router_softmax_top_gb300 as moe
from oracle import fp4_oracle as Q
from oracle import fp8_oracle as O8

pytestmark = pytest.mark.gpu
BF, U8, E4 = torch.bfloat16, torch.uint8, torch.float8_e4m3fn
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def built():
    from combine_router_softmax_top_gb300 import build
    build.build()


def f64(t):
    return t.detach().double().cpu().numpy()


def rnd(*s, std=1.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*s, generator=g, device="cuda") * std).to(BF)


def desc(T, H):
    return moe.LayerDesc.of(T, H, 1, 1, 64)


def words(T, H):
    return torch.full((-(-H // 512), max(T, 1), 4), 0x5A, dtype=U8, device="cuda")


def forward(T, H, residual=True, q8=True, y=True, seed=0, eps=EPS, x=None):
    x = rnd(T, H, seed=seed) if x is None else x
    res = rnd(T, H, std=3, seed=seed + 1) if residual else None
    w = (1 + 0.2 * rnd(H, seed=seed + 2).float()).to(BF)
    pad = lambda dt: torch.full((T + 1, H), 7.0, device="cuda").to(dt)  # noqa: E731
    out = dict(r=pad(BF) if residual else None, y=pad(BF) if y else None, yq=pad(E4) if q8 else None,
               ys=words(T, H) if q8 else None, rstd=torch.full((T + 1,), 7.0, device="cuda"))
    moe.moe_rms_norm(desc(T, H), x, res, w, eps, out["r"], out["y"], out["yq"], out["ys"], out["rstd"])
    return x, res, w, out


SHAPES = [(1, 64), (1, 2048), (1, 16384), (2, 320), (3, 128), (5, 192), (7, 704), (130, 2048),
          (607, 64), (609, 576), (700, 320), (1000, 1024), (2000, 128), (650, 4096), (700, 5056),
          (640, 8256), (620, 16384), (5000, 192), (4096, 2048)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("residual,q8", [(True, True), (False, True), (True, False)])
def test_forward(T, H, residual, q8):
    x, res, w, out = forward(T, H, residual, q8, seed=T + H)
    total = f64(x) + (f64(res) if residual else 0)
    if residual:
        r = f64(out["r"])
        assert (r[T:] == 7).all()
        r = r[:T]
        assert (np.abs(r - total) <= np.abs(total) * (2.0 ** -8 + 2.0 ** -23)).all()
    else:
        r = total
    y, rstd = Q.rms_norm(r, f64(w), EPS)
    e = (H / 2 + 8) * 2.0 ** -24
    got = f64(out["rstd"])
    assert got[T] == 7 and (np.abs(got[:T] - rstd) <= e * rstd).all()
    yv = f64(out["y"])
    assert (yv[T:] == 7).all()
    assert (np.abs(yv[:T] - y) <= np.abs(y) * (2.0 ** -8 + 2 * e) + 1e-38).all()
    if q8:  # the bits that the 8-bit permute makes of y
        d = desc(T, H)
        q, s = torch.empty(T, H, dtype=E4, device="cuda"), words(T, H)
        moe.moe_permute_fp8(d, out["y"][:T].contiguous(), torch.arange(T, dtype=torch.int32, device="cuda"), q, s)
        assert torch.equal(out["yq"][:T].view(U8), q.view(U8)) and (out["yq"][T:].float() == 7).all()
        assert torch.equal(out["ys"], s)
        if T * H < 100000:
            qv, b = O8.quantize_rows(yv[:T])
            assert (f64(out["yq"])[:T] == qv).all()
            assert (O8.unpack_words(out["ys"].cpu().numpy(), b.shape[1]) == b).all()


@pytest.mark.parametrize("T,H", [(3, 320), (900, 320), (900, 2048)])
def test_which_outputs_are_asked_for_changes_nothing(T, H):
    x, res, w, full = forward(T, H)
    d = desc(T, H)
    yq, ys, y = torch.empty(T, H, dtype=E4, device="cuda"), words(T, H), torch.empty(T, H, dtype=BF, device="cuda")
    moe.moe_rms_norm(d, x, res, w, EPS, None, None, yq, ys)
    assert torch.equal(yq.view(U8), full["yq"][:T].view(U8)) and torch.equal(ys, full["ys"])
    moe.moe_rms_norm(d, x, res, w, EPS, None, y)
    assert torch.equal(y, full["y"][:T])
    for inplace in (x.clone(), res.clone()):  # the stream updated in place
        a, b = (inplace, res) if torch.equal(inplace, x) else (x, inplace)
        y.zero_()
        moe.moe_rms_norm(d, a, b, w, EPS, inplace, y)
        assert torch.equal(inplace, full["r"][:T]) and torch.equal(y, full["y"][:T])


@pytest.mark.parametrize("T", [4, 800])
def test_special_rows(T):
    H = 320
    x = rnd(T, H, seed=3)
    x[0] = 0
    x[1, 5] = float("nan")
    x[2, 300] = float("inf")
    x[3] = 2.0 ** -60  # squares far below 1e-6
    _, _, w, out = forward(T, H, residual=False, x=x)
    y, s = out["y"][:T], out["ys"].cpu().numpy()
    assert (y[0] == 0).all() and torch.isnan(y[1]).all()
    assert torch.isnan(y[2, 300]) and (y[2, :300] == 0).all()  # inf / inf, and the rest over inf
    want = 2.0 ** -60 / np.sqrt(2.0 ** -120 + EPS) * f64(w)
    assert (np.abs(f64(y[3]) - want) <= np.abs(want) * 2.0 ** -7).all()
    b = O8.unpack_words(s, 3)
    assert (b[1] == 255).all() and b[2].tolist() == [0, 0, 255] and (b[0] == 0).all()
    if T > 4:
        assert torch.isfinite(y[4:].float()).all()


def backward(T, H, residual=True, seed=0):
    dy, dr = rnd(T, H, seed=seed), rnd(T, H, seed=seed + 1) if residual else None
    r, w = rnd(T, H, std=2, seed=seed + 2), (1 + 0.2 * rnd(H, seed=seed + 3).float()).to(BF)
    rstd = torch.rsqrt(r.float().square().mean(1) + EPS)
    d = desc(T, H)
    ws = torch.full((moe.moe_rms_norm_bwd_workspace_size(d),), 0xFF, dtype=U8, device="cuda")
    dx = torch.full((T + 1, H), 7.0, dtype=BF, device="cuda")
    dw = torch.full((H + 4,), 7.0, device="cuda")
    return d, dy, dr, r, w, rstd, dx, dw, ws


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("residual", [True, False])
def test_backward(T, H, residual):
    d, dy, dr, r, w, rstd, dx, dw, ws = backward(T, H, residual, seed=T + H)
    moe.moe_rms_norm_bwd(d, dy, dr, r, w, rstd, dx, dw, ws)
    args = [f64(t) for t in (dy, r, w, rstd)]
    want, want_w = Q.rms_norm_bwd(*args, f64(dr) if residual else None)
    xh = np.abs(args[1] * args[3][:, None])
    g = np.abs(args[0] * args[2])
    dot = (g * xh).sum(1, keepdims=True) / H
    e = args[3][:, None] * (8 * 2.0 ** -24 * (g + xh * dot) + (H + 8) * 2.0 ** -24 * xh * dot)
    e = e + 2.0 ** -23 * (np.abs(want) + (np.abs(f64(dr)) if residual else 0))
    got = f64(dx)
    assert (got[T:] == 7).all()
    assert (np.abs(got[:T] - want) <= e + (np.abs(want) + e) * 2.0 ** -8).all()
    ew = (T + 4) * 2.0 ** -24 * (np.abs(args[0]) * xh).sum(0)
    gw = f64(dw)
    assert (gw[H:] == 7).all() and (np.abs(gw[:H] - want_w) <= ew).all()


@pytest.mark.parametrize("T,H", [(5, 128), (3000, 320)])
def test_backward_repeats_itself_and_works_in_place(T, H):
    d, dy, dr, r, w, rstd, dx, dw, ws = backward(T, H)
    moe.moe_rms_norm_bwd(d, dy, dr, r, w, rstd, dx, dw, ws)
    x1, w1 = dx[:T].clone(), dw.clone()
    for target in (dy.clone(), dr.clone()):
        a, b = (target, dr) if torch.equal(target, dy) else (dy, target)
        ws.fill_(0x7F)
        moe.moe_rms_norm_bwd(d, a, b, r, w, rstd, target, dw, ws)
        assert torch.equal(target, x1) and torch.equal(dw, w1)


def test_no_tokens():
    H = 192
    d = desc(0, H)
    z = lambda *s, dt=BF: torch.full(s, 7.0, device="cuda").to(dt)  # noqa: E731
    x, y, dw, rstd = z(1, H), z(1, H), z(H, dt=torch.float32), z(1, dt=torch.float32)
    ws = torch.zeros(moe.moe_rms_norm_bwd_workspace_size(d), dtype=U8, device="cuda")
    moe.moe_rms_norm(d, x, None, z(H), EPS, None, y, None, None, rstd)
    moe.moe_rms_norm_bwd(d, x, None, x, z(H), rstd, y, dw, ws)
    assert (y == 7).all() and (rstd == 7).all() and (dw == 0).all()


def test_rows_past_32_bits():
    T, H = 1 << 18, 16384  # 2^32 elements
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    x = torch.ones(T, H, dtype=BF, device="cuda")
    x[-3:] = rnd(3, H, seed=1)
    w = (1 + 0.2 * rnd(H, seed=2).float()).to(BF)
    y, rstd = torch.zeros_like(x), torch.zeros(T, device="cuda")
    moe.moe_rms_norm(desc(T, H), x, None, w, EPS, None, y, None, None, rstd)
    small, small_r = torch.zeros(3, H, dtype=BF, device="cuda"), torch.zeros(3, device="cuda")
    moe.moe_rms_norm(desc(3, H), x[-3:].contiguous(), None, w, EPS, None, small, None, None, small_r)
    # (another split of the row into threads: another order of the sum)
    assert (np.abs(f64(rstd[-3:]) / f64(small_r) - 1) < (H + 16) * 2.0 ** -24).all()
    assert (np.abs(f64(y[-3:]) - f64(small)) <= np.abs(f64(small)) * 2.0 ** -7).all()
    assert (y[1000] == w).all() and (y[-4] == w).all()


@pytest.mark.parametrize("T,H", [(2, 2048), (900, 320)])
def test_streams_and_captures(T, H):
    x, res, w, full = forward(T, H)
    d, dy, dr, r, wb, rstd, dx, dw, ws = backward(T, H)
    moe.moe_rms_norm_bwd(d, dy, dr, r, wb, rstd, dx, dw, ws)
    want = (full["y"].clone(), dx.clone(), dw.clone())
    y = full["y"]
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    y.fill_(7), dx.fill_(7), dw.fill_(7)
    torch.cuda.synchronize()
    moe.moe_rms_norm(d, x, res, w, EPS, full["r"], y, stream=st)
    moe.moe_rms_norm_bwd(d, dy, dr, r, wb, rstd, dx, dw, ws, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(y, want[0]) and torch.equal(dx, want[1]) and torch.equal(dw, want[2])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_rms_norm(d, x, res, w, EPS, full["r"], y)
        moe.moe_rms_norm_bwd(d, dy, dr, r, wb, rstd, dx, dw, ws)
    for _ in range(3):
        y.fill_(7), dx.fill_(7), dw.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(dx, want[1]) and torch.equal(dw, want[2])


def test_refuses_wrong_tensors():
    T, H = 4, 128
    x, res, w, out = forward(T, H)
    args = [x, res, w, EPS, out["r"], out["y"], out["yq"], out["ys"], out["rstd"]]
    for i, bad, why in ((0, x.float(), "float32"), (0, rnd(H, T).t(), "contiguous"), (1, res[:2], "fewer"),
                        (2, w[:64], "fewer"), (5, out["y"].cpu(), "device"), (6, out["yq"].view(U8), "uint8"),
                        (7, out["ys"].flatten()[:15].contiguous(), "fewer"), (8, out["rstd"].half(), "float16")):
        with pytest.raises(moe.MoeError, match=why):
            moe.moe_rms_norm(desc(T, H), *[bad if j == i else t for j, t in enumerate(args)])


def test_an_always_on_expert_on_the_norms_rows():
    """norm with 8-bit rows -> the 8-bit expert products of one expert that every token visits."""
    T, H, F = 90, 320, 192
    d = moe.LayerDesc.of(T, H, 1, 1, F)
    x, res, w, out = forward(T, H)
    f = moe.Fp8Buffers(d, backward=False)
    f.quantize_weights(rnd(1, 2 * F, H, std=0.1, seed=5), rnd(1, H, F, std=0.1, seed=6))
    ws = torch.zeros(moe.moe_workspace_size(d), dtype=U8, device="cuda")
    off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    outs = []
    for q, s in ((out["yq"], out["ys"]), (f.xq, f.xs)):
        if q is f.xq:
            moe.moe_permute_fp8(d, out["y"], torch.arange(T, dtype=torch.int32, device="cuda"), q, s)
        o = torch.zeros(T, H, dtype=BF, device="cuda")
        moe.moe_expert_ffn_fwd_fp8(d, q, s, off, f.w1q, f.w1s, f.w2q, f.w2s, None, None, f.hq, f.hs, o, ws)
        outs.append(o)
    assert moe.moe_device_status(d, ws) == moe.MOE_OK
    assert torch.equal(*outs) and outs[0].abs().max() > 0


@pytest.mark.parametrize("T", [3, 400])
def test_norm_into_the_layer_and_back(T):
    """A pre-norm block as it is trained: norm, 4-bit layer forward, backward, norm gradient.
    The block's dx from the layer's own dx in float64."""
    H, E, k, F = 256, 8, 2, 128
    d = moe.LayerDesc.of(T, H, E, k, F)
    b, f = moe.LayerBuffers(d), moe.Fp4Buffers(d)
    b.w_r.copy_(rnd(E, H, std=0.1, seed=2))
    f.quantize_weights(rnd(E, 2 * F, H, std=0.1, seed=3), rnd(E, H, F, std=0.1, seed=4), b.w1, b.w2)
    x, res = rnd(T, H, seed=5), rnd(T, H, seed=6)
    w = (1 + 0.2 * rnd(H, seed=7).float()).to(BF)
    r, rstd = torch.empty(T, H, dtype=BF, device="cuda"), torch.empty(T, device="cuda")
    moe.moe_rms_norm(d, x, res, w, EPS, r, b.x, rstd=rstd)
    moe.moe_layer_forward_fp4(d, b, f, save=True)
    out = r.float() + b.y.float()
    dout = rnd(T, H, seed=8)  # of the block's output: of r directly, and of y
    b.dy.copy_(dout)
    moe.moe_layer_backward(d, b)
    dx, dw = torch.empty(T, H, dtype=BF, device="cuda"), torch.empty(H, device="cuda")
    ws = torch.zeros(moe.moe_rms_norm_bwd_workspace_size(d), dtype=U8, device="cuda")
    moe.moe_rms_norm_bwd(d, b.dx, dout, r, w, rstd, dx, dw, ws)
    assert moe.moe_device_status(d, b.ws) == moe.MOE_OK and torch.isfinite(out).all()
    want, want_w = Q.rms_norm_bwd(f64(b.dx), f64(r), f64(w), f64(rstd), f64(dout))
    xh, g = np.abs(f64(r) * f64(rstd)[:, None]), np.abs(f64(b.dx) * f64(w))
    dot = (g * xh).sum(1, keepdims=True) / H
    e = f64(rstd)[:, None] * (8 * 2.0 ** -24 * g + (H + 16) * 2.0 ** -24 * xh * dot) + 2.0 ** -23 * (np.abs(want) + np.abs(f64(dout)))
    assert (np.abs(f64(dx) - want) <= e + (np.abs(want) + e) * 2.0 ** -8).all()
    assert (np.abs(f64(dw) - want_w) <= (T + 4) * 2.0 ** -24 * (np.abs(f64(b.dx)) * xh).sum(0) + 1e-38).all()
