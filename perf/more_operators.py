"""What the layer's input norm and its 4-bit floating-point experts are measured on.

  norm        the residual's addition and root-mean-square norm in front of the layer, its result
              in bf16 and, for an always-on expert, as e4m3 rows with one scale for each 128 columns;
  norm_grad   its gradient: with respect to the sum and to the norm's weights;
  weights     the experts' bf16 weights into microscaled 4-bit values (e2m1, two a byte, one
              power-of-two scale for each 32 along K) and the bf16 values that those stand for;
  experts     tokens to expert outputs on such operands: the permute that quantises, the two grouped
              products with SwiGLU between them.

run() computes them in plain torch operations, or, with `own` set, through the package's entry points.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # magnitudes of e2m1, by code


# ----------------------------------------------------------------------------- cases
def _norm(name, T, H, q8=False, train=False, residual=True, op="norm"):
    return {"name": name, "op": op, "T": T, "H": H, "q8": q8, "train": train, "residual": residual}


def _experts(name, op, T, H, E, k, F, routing="balanced", train=False):
    return {"name": name, "op": op, "T": T, "H": H, "E": E, "k": k, "F": F,
            "routing": routing, "train": train}


def listed():
    return [
        # one token of a decode step, with 8-bit rows for the always-on expert: latency alone
        _norm("norm_one_token", 1, 2048, q8=True),
        # a training micro-batch: the sum and the reciprocal norms are kept for the gradient
        _norm("norm_layer", 4096, 2048, train=True),
        # a batch of long prompts, served with 8-bit rows
        _norm("norm_prompts", 32768, 2048, q8=True),
        # odd sizes, at the first layer: no residual gradient joins
        _norm("norm_grad_ragged", 1000, 320, residual=False, op="norm_grad"),
        # a training micro-batch, the residual stream's gradient added
        _norm("norm_grad_layer", 4096, 2048, op="norm_grad"),
        # the smallest layer's weights, then the 128-expert layer's: laid out after an optimizer step
        _experts("weights_small", "weights", 1, 128, 8, 2, 256),
        _experts("weights_layer", "weights", 1, 2048, 128, 8, 768),
        # serving one token: eight experts with one row each
        _experts("experts_one_token", "experts", 1, 2048, 128, 8, 768),
        # serving a batch of 64 sequences, one token each: every expert has a few rows
        _experts("experts_decode_batch", "experts", 64, 2048, 128, 8, 768, "skewed"),
        # odd sizes, experts of a few rows next to experts of hundreds; kept for a backward
        _experts("experts_ragged", "experts", 1000, 320, 16, 4, 448, "skewed", True),
        # training forward: the pre-activation and h are stored for the backward
        _experts("experts_train", "experts", 4096, 2048, 128, 8, 768, "balanced", True),
        # prompts on the 64-expert layer: a thousand rows an expert, and many more at some
        _experts("experts_prefill", "experts", 8192, 2048, 64, 8, 1408, "skewed"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "norm_grad", "weights", "experts", "experts"))
    if op.startswith("norm"):
        H = 64 * _log(rng, 1, 64)
        return {"op": op, "T": _log(rng, 1, max(1, min(32768, (32768 * 2048) // H))), "H": H,
                "q8": rng.random() < 0.5 and op == "norm", "train": rng.random() < 0.5,
                "residual": rng.random() < 0.7}
    H = 64 * _log(rng, 1, 32)
    F = 64 * _log(rng, 1, 22)
    E = max(1, min(_log(rng, 1, 128), (128 * 768 * 2048) // (F * H)))
    k = rng.randint(1, min(8, E))
    T = 1 if op == "weights" else _log(rng, 1, 8192)
    return {"op": op, "T": T, "H": H, "E": E, "k": k, "F": F,
            "routing": rng.choice(("balanced", "skewed")), "train": rng.random() < 0.5}


def _skew(E, rank):
    """What skewed routing adds to the logits of the experts of these popularity ranks (1 .. E)."""
    w = rank ** -1.1
    return -3 + 6 * (w - E ** -1.1) / (1 - E ** -1.1 + 1e-9)


def _used(case):
    """Experts that some token picks."""
    T, E, k = case["T"], case["E"], case["k"]
    if case["routing"] == "balanced" or T > 512:
        return min(E, T * k)
    z = np.random.RandomState(0).randn(8, T, E) * 0.9 + _skew(E, np.arange(E) + 1.0)
    picked = np.argsort(-z, 2)[:, :, :k].reshape(8, -1)
    return float(np.mean([len(np.unique(p)) for p in picked]))


def work(case):
    T, H = case["T"], case["H"]
    if case["op"] == "norm":
        streams = 2.0 * T * H * (4 if case["residual"] else 2)  # x, y, and the other addend and the sum
        return {"bytes": streams + 2 * H + (T * (H + math.ceil(H / 128)) if case["q8"] else 0)
                + (4 * T if case["train"] else 0), "flops": 6.0 * T * H}
    if case["op"] == "norm_grad":
        return {"bytes": 2.0 * T * H * (4 if case["residual"] else 3) + 4 * T + 6 * H,
                "flops": 10.0 * T * H}
    E, k, F = case["E"], case["k"], case["F"]
    if case["op"] == "weights":
        n = 3.0 * E * F * H
        return {"bytes": 2 * n + n * 17 / 32 + 2 * n, "flops": 3 * n}
    N = T * k
    rows = 2.0 * T * H + 4 * N + 2.0 * N * H + (6.0 * N * F if case["train"] else 0)
    return {"bytes": _used(case) * 3.0 * F * H * 17 / 32 + rows + 4 * (E + 1),
            "flops": 6.0 * N * F * H}


# ----------------------------------------------------------------------------- inputs
def _route(case, g, dev):
    """off [E + 1], slot [T, k] of a routing drawn from g, and the largest expert's rows."""
    T, E, k = case["T"], case["E"], case["k"]
    if case["routing"] == "balanced":
        idx = (k * torch.arange(T, device=dev)[:, None] + torch.arange(k, device=dev)) % E
    else:
        rank = torch.randperm(E, generator=g, device=dev) + 1.0
        z = torch.randn(T, E, generator=g, device=dev) * 0.9 + _skew(E, rank)
        idx = z.topk(k, 1).indices
    cnt = torch.bincount(idx.flatten(), minlength=E)
    off = torch.cat([cnt.new_zeros(1), cnt.cumsum(0)])
    slot = torch.empty(T * k, dtype=torch.int64, device=dev)
    slot[torch.sort(idx.flatten(), stable=True).indices] = torch.arange(T * k, device=dev)
    return off.to(torch.int32), slot.view(T, k).to(torch.int32), int(cnt.max())


def prepare(case, seed):
    dev, bf, u8 = "cuda", torch.bfloat16, torch.uint8
    T, H = case["T"], case["H"]
    g = torch.Generator(device=dev).manual_seed(seed)
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=g, device=dev) * std).to(bf)  # noqa: E731
    new = lambda *s, dt=bf: torch.empty(*s, dtype=dt, device=dev)  # noqa: E731
    s = {"case": dict(case)}
    if case["op"].startswith("norm"):
        s["w"] = (1 + 0.1 * torch.randn(H, generator=g, device=dev)).to(bf)
        # a residual stream: a few columns far larger than the others
        scale = torch.exp(0.7 * torch.randn(H, generator=g, device=dev))
        stream = (torch.randn(T, H, generator=g, device=dev) * scale).to(bf)
        if case["op"] == "norm":
            s["x"], s["res"] = (rnd(T, H), stream) if case["residual"] else (stream, None)
            s["r"] = new(T, H) if case["residual"] else None
            s["y"] = new(T, H)
            s["yq"] = new(T, H, dt=torch.float8_e4m3fn) if case["q8"] else None
            s["ys"] = new(-(-H // 512), T, 4, dt=u8) if case["q8"] else None
            s["rstd"] = new(T, dt=torch.float32) if case["train"] else None
        else:
            s["r"], s["dy"] = stream, rnd(T, H, std=0.02)
            s["rstd"] = torch.rsqrt(stream.float().square().mean(1) + EPS)
            s["dr"] = rnd(T, H, std=0.02) if case["residual"] else None
            s["dx"], s["dw"] = new(T, H), new(H, dt=torch.float32)
        return s
    E, k, F = case["E"], case["k"], case["F"]
    gh, gf = -(-H // 256), -(-F // 256)
    w1, w2 = rnd(E, 2 * F, H, std=0.02), rnd(E, H, F, std=0.02)
    if case["op"] == "weights":
        s["w1"], s["w2"] = w1, w2
        s["w1q"], s["w2q"] = new(E, 2 * F, H // 2, dt=u8), new(E, H, F // 2, dt=u8)
        s["w1s"], s["w2s"] = new(E, 2, gh, F, 8, dt=u8), new(E, gf, H, 8, dt=u8)
        s["w1v"], s["w2v"] = new(E, 2 * F, H), new(E, H, F)
        return s
    N = T * k
    s["off"], s["slot"], s["rows_max"] = _route(case, g, dev)
    s["x"] = rnd(T, H)
    q, b = _quantize(w1.float())
    s["w1q"], s["w1s"] = _pack(q), _groups(b.view(E, 2, F, -1))
    q, b = _quantize(w2.float())
    s["w2q"], s["w2s"] = _pack(q), _groups(b)
    even = (N + 1) // 2 * 2
    s["xq"], s["xs"] = new(N, H // 2, dt=u8), new(gh, even, 8, dt=u8)
    s["hq"], s["hs"] = new(N, F // 2, dt=u8), new(gf, even, 8, dt=u8)
    s["a"] = new(N, 2 * F) if case["train"] else None
    s["h"] = new(N, F) if case["train"] else None
    s["o"] = new(N, H)
    return s


# ----------------------------------------------------------------------------- plain forms
def _quantize(x):
    """fp32 [..., C] -> e2m1 codes [..., C] and scale bytes [..., C / 32]: the smallest power of two
    that brings the block's largest value to 6 or below; ties to the even code."""
    y = x.unflatten(-1, (-1, 32))
    b = ((y.abs().amax(-1).view(torch.int32) + 0x3FFFFF) >> 23).sub(2).clamp(min=0)
    y = y * ((254 - b) << 23).view(torch.float32).unsqueeze(-1)
    m = y.abs()
    # codes step by 1/2 up to 2, by 1 up to 4, by 2 up to 6; rounding is to even in each
    code = torch.where(m < 2, torch.round(2 * m),
                       torch.where(m < 4, torch.round(m) + 2, torch.round(m / 2) + 4))
    code = (code + 8 * torch.signbit(y)).to(torch.uint8)
    return code.flatten(-2), b.to(torch.uint8)


def _values(code, b):
    """What codes [..., C] with scale bytes [..., C / 32] stand for, fp32."""
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device=code.device)
    v = grid[code.int()].unflatten(-1, (-1, 32))
    return (v * (b.int() << 23).view(torch.float32).unsqueeze(-1)).flatten(-2)


def _pack(code):
    """Two codes a byte, the lower column in the low bits."""
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _unpack(q):
    return torch.stack((q & 15, q >> 4), -1).flatten(-2)


def _groups(b):
    """Scale bytes [..., R, nb] -> [..., ceil(nb / 8), R, 8]: the eight of 256 columns side by side."""
    nb = b.shape[-1]
    b = torch.nn.functional.pad(b, (0, -nb % 8))
    return b.unflatten(-1, (-1, 8)).transpose(-3, -2).contiguous()


def _ungroup(s, nb):
    return s.transpose(-3, -2).flatten(-2)[..., :nb]


def _grouped(rows, w, off, rows_max):
    """rows[s] @ w[expert of s]^T, fp32: [N, K], [E, M, K] -> [N, M]."""
    N, E = rows.shape[0], w.shape[0]
    s = torch.arange(N, device=rows.device)
    e = torch.searchsorted(off[1:].contiguous(), s.to(off.dtype), right=True)
    if 2 * N <= E:  # few rows: each with its own expert's weights
        return torch.bmm(w[e], rows.unsqueeze(2)).squeeze(2)
    at = (off[:-1, None] + torch.arange(rows_max, device=rows.device)).clamp(max=N - 1).long()
    return torch.bmm(rows[at], w.transpose(1, 2))[e, s - off[e].long()]


def _plain_norm(s):
    c, bf = s["case"], torch.bfloat16
    w = s["w"].float()
    if c["op"] == "norm_grad":
        dy, rstd = s["dy"].float(), s["rstd"].unsqueeze(1)
        xh = s["r"].float() * rstd
        gy = dy * w
        dx = rstd * (gy - xh * (gy * xh).mean(1, keepdim=True))
        if s["dr"] is not None:
            dx = dx + s["dr"].float()
        return {"dx": dx.to(bf), "dw": (dy * xh).sum(0)}
    r = s["x"] if s["res"] is None else (s["x"].float() + s["res"].float()).to(bf)
    rf = r.float()
    rstd = 1 / torch.sqrt(rf.square().mean(1) + EPS)
    y = (rf * rstd.unsqueeze(1) * w).to(bf)
    out = {"y": y}
    if c["residual"]:
        out["r"] = r
    if c["train"]:
        out["rstd"] = rstd
    if c["q8"]:
        C = y.shape[1]
        v = torch.nn.functional.pad(y.float(), (0, -C % 128)).unflatten(1, (-1, 128))
        b = ((v.abs().amax(2).view(torch.int32) + 0x1FFFFF) >> 23).sub(8).clamp(min=0)
        q = (v * ((254 - b) << 23).view(torch.float32).unsqueeze(2)).to(torch.float8_e4m3fn)
        b = torch.nn.functional.pad(b, (0, -b.shape[1] % 4)).to(torch.uint8)
        words = b.unflatten(1, (-1, 4)).transpose(0, 1).contiguous()
        out["yq"] = q.flatten(1)[:, :C].contiguous()
        out["ys"] = words.view(torch.float8_e8m0fnu)
    return out


def _plain(s):
    c, bf = s["case"], torch.bfloat16
    if c["op"].startswith("norm"):
        return _plain_norm(s)
    E, F, H = c["E"], c["F"], c["H"]
    if c["op"] == "weights":
        q1, b1 = _quantize(s["w1"].float())
        q2, b2 = _quantize(s["w2"].float())
        return {"w1q": _pack(q1), "w2q": _pack(q2),
                "w1s": _groups(b1.view(E, 2, F, -1)).view(torch.float8_e8m0fnu),
                "w2s": _groups(b2).view(torch.float8_e8m0fnu),
                "w1v": _values(q1, b1).to(bf), "w2v": _values(q2, b2).to(bf)}
    x = _values(*_quantize(s["x"].float()))
    row = torch.empty(s["slot"].numel(), dtype=torch.int64, device=x.device)
    row[s["slot"].flatten().long()] = torch.arange(row.numel(), device=x.device) // c["k"]
    w1 = _values(_unpack(s["w1q"]), _ungroup(s["w1s"], H // 32).flatten(1, 2))
    w2 = _values(_unpack(s["w2q"]), _ungroup(s["w2s"], F // 32))
    a = _grouped(x[row], w1, s["off"], s["rows_max"])
    ag, au = a.chunk(2, 1)
    h = ag * torch.sigmoid(ag) * au
    o = _grouped(_values(*_quantize(h)), w2, s["off"], s["rows_max"]).to(bf)
    return {"a": a.to(bf), "h": h.to(bf), "o": o} if c["train"] else {"o": o}


def run(state):
    if not own:
        return _plain(state)
    import combine_router_softmax_top_gb300 as moe
    s, c = state, state["case"]
    op = c["op"]
    if "desc" not in s:  # a program keeps its descriptor and workspace
        if op.startswith("norm"):
            s["desc"] = moe.LayerDesc.of(c["T"], c["H"], 1, 1, 64)
            n = moe.moe_rms_norm_bwd_workspace_size(s["desc"])
        else:
            s["desc"] = moe.LayerDesc.of(c["T"], c["H"], c["E"], c["k"], c["F"])
            n = moe.moe_workspace_size(s["desc"])
        s["ws"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
    d = s["desc"]
    scales = torch.float8_e8m0fnu
    if op == "norm":
        moe.moe_rms_norm(d, s["x"], s["res"], s["w"], EPS, s["r"], s["y"], s["yq"], s["ys"],
                         s["rstd"])
        out = {n: s[n] for n in ("r", "y", "yq", "rstd") if s[n] is not None}
        if c["q8"]:
            out["ys"] = s["ys"].view(scales)
        return out
    if op == "norm_grad":
        moe.moe_rms_norm_bwd(d, s["dy"], s["dr"], s["r"], s["w"], s["rstd"], s["dx"], s["dw"],
                             s["ws"])
        return {"dx": s["dx"], "dw": s["dw"]}
    if op == "weights":
        moe.moe_fp4_quantize_weights(d, s["w1"], s["w2"], s["w1q"], s["w1s"], s["w2q"], s["w2s"],
                                     s["w1v"], s["w2v"])
        return {"w1q": s["w1q"], "w2q": s["w2q"], "w1s": s["w1s"].view(scales),
                "w2s": s["w2s"].view(scales), "w1v": s["w1v"], "w2v": s["w2v"]}
    moe.moe_permute_fp4(d, s["x"], s["slot"], s["xq"], s["xs"])
    moe.moe_expert_ffn_fwd_fp4(d, s["xq"], s["xs"], s["off"], s["w1q"], s["w1s"], s["w2q"],
                               s["w2s"], s["a"], s["h"], s["hq"], s["hs"], s["o"], s["ws"])
    return {n: s[n] for n in ("a", "h", "o") if s[n] is not None}


# ----------------------------------------------------------------------------- in 64 bits
def _nearest(x, grid, block, top):
    """x (float64) rounded under one power-of-two scale for each `block` columns, by distance to every
    value of `grid` (ties to the even place in it), and the scales; `top` is the largest value."""
    y = torch.nn.functional.pad(x, (0, -x.shape[-1] % block)).unflatten(-1, (-1, block))
    amax = y.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(amax > 0, amax, 1.0) / top))
    e = torch.where(amax > top * torch.exp2(e), e + 1, e)  # log2 may be off next to an integer
    e = torch.where(amax <= top * torch.exp2(e - 1), e - 1, e)
    e = torch.where(amax > 0, e, -127.0).clamp(min=-127)
    m = (y * torch.exp2(-e)).abs()
    mid = (grid[:-1] + grid[1:]) / 2
    lo, hi = torch.searchsorted(mid, m), torch.searchsorted(mid, m, right=True)
    at = torch.where(lo == hi, lo, torch.where(lo % 2 == 0, lo, hi))
    v = torch.where(y < 0, -1.0, 1.0) * grid[at] * torch.exp2(e)
    return v.flatten(-2)[..., : x.shape[-1]], e


def exact(case, seed):
    # what the operators hold in bf16, 8 or 4 bits on the way is rounded here too; results are not
    s = prepare(case, seed)
    rd = lambda t: t.to(torch.bfloat16).double()  # noqa: E731
    dev = "cuda"
    if case["op"] == "norm_grad":
        # dx = rstd (I - xh xh^T / H) (w dy) + dr, with xh of the kept rstd
        H = case["H"]
        r, dy, rs = s["r"].double(), s["dy"].double(), s["rstd"].double()[:, None]
        c = (dy * s["w"].double() * r).sum(1, keepdim=True) * rs * rs / H
        dx = rs * (dy * s["w"].double() - r * c)
        return {"dx": dx if s["dr"] is None else dx + s["dr"].double(),
                "dw": torch.einsum("th,th,t->h", dy, r, rs[:, 0])}
    if case["op"] == "norm":
        total = s["x"].double() + (0 if s["res"] is None else s["res"].double())
        r = rd(total)
        ms = torch.einsum("th,th->t", r, r) / case["H"] + EPS
        y = r * s["w"].double() / ms.sqrt()[:, None]
        out = {"y": y}
        if case["residual"]:
            out["r"] = total
        if case["train"]:
            out["rstd"] = ms ** -0.5
        if case["q8"]:
            e4m3 = torch.arange(127, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn).double()
            v, e = _nearest(rd(y), e4m3, 128, 448.0)
            out["yq"] = v * torch.exp2(-e).squeeze(-1).repeat_interleave(128, 1)[:, : case["H"]]
            out["ys"] = None
        return out
    e2m1 = torch.tensor(GRID, dtype=torch.float64, device=dev)
    E, F, H, k = case["E"], case["F"], case["H"], case["k"]
    if case["op"] == "weights":
        out = {"w1q": None, "w2q": None, "w1s": None, "w2s": None}
        for n in ("w1", "w2"):
            out[n + "v"] = torch.stack([_nearest(w.double(), e2m1, 32, 6.0)[0] for w in s[n]])
        return out

    def matrix(q, b):
        """One matrix of packed codes and [groups, R, 8] scale bytes, as values."""
        R, half = q.shape
        v = torch.empty(R, 2 * half, dtype=torch.float64, device=dev)
        for i in (0, 1):
            c = (q >> (4 * i)) & 15
            v[:, i::2] = torch.where(c > 7, -1.0, 1.0) * e2m1[(c & 7).long()]
        sc = b.permute(1, 0, 2).reshape(R, -1)[:, : 2 * half // 32].double()
        return v * torch.exp2(sc - 127).repeat_interleave(32, 1)

    slot = s["slot"].flatten().long()
    N = slot.numel()
    x = torch.empty(N, H, dtype=torch.float64, device=dev)
    x[slot] = _nearest(s["x"].double(), e2m1, 32, 6.0)[0].repeat_interleave(k, 0)
    a = torch.empty(N, 2 * F, dtype=torch.float64, device=dev)
    o = torch.empty(N, H, dtype=torch.float64, device=dev)
    off = s["off"].tolist()
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        for i in (0, 1):
            w = matrix(s["w1q"][e, i * F : (i + 1) * F], s["w1s"][e, i])
            a[lo:hi, i * F : (i + 1) * F] = x[lo:hi] @ w.T
        h = a[lo:hi, :F] / (1 + torch.exp(-a[lo:hi, :F])) * a[lo:hi, F:]
        o[lo:hi] = _nearest(h, e2m1, 32, 6.0)[0] @ matrix(s["w2q"][e], s["w2s"][e]).T
    if not case["train"]:
        return {"o": o}
    return {"a": a, "h": a[:, :F] / (1 + torch.exp(-a[:, :F])) * a[:, F:], "o": o}
