"""Host-side checks of the 4-bit experts and of the input norm (no GPU work): the C entry
points and the binding refuse bad arguments before anything is launched."""
import ctypes

import pytest
import torch

import combine_router_softmax_top_gb300 as moe
from combine_router_softmax_top_gb300 import build


@pytest.fixture(scope="module")
def L():
    build.build()
    return moe.lib()


P = ctypes.c_void_p(4096)
D = moe.LayerDesc.of(T=16, H=192, E=8, k=2, F=192)
BAD = moe.LayerDesc.of(T=16, H=100, E=8, k=2, F=192)

# entry point -> (its pointer arguments after the descriptor, which of them may be NULL)
CALLS = {
    "moe_fp4_quantize_weights": (8, (6, 7)),
    "moe_permute_fp4": (4, ()),
    "moe_expert_ffn_fwd_fp4": (13, (7, 8)),
    "moe_rms_norm": (8, (1, 3, 4, 5, 6, 7)),
    "moe_rms_norm_bwd": (8, (1,)),
}


def call(L, name, args, desc=D, ws_bytes=1 << 30, eps=1e-6):
    args = list(args)
    if name == "moe_rms_norm":
        args.insert(3, ctypes.c_float(eps))
    if name in ("moe_expert_ffn_fwd_fp4", "moe_rms_norm_bwd"):
        args.append(ws_bytes)
    return getattr(L, name)(None if desc is None else ctypes.byref(desc), *args, None)


@pytest.mark.parametrize("name", sorted(CALLS))
def test_null_and_misaligned_pointers(L, name):
    n, optional = CALLS[name]
    for i in range(n):
        args = [P] * n
        if i not in optional:
            args[i] = None
            assert call(L, name, args) == moe.MOE_ERR_INVALID_ARG, i
            assert b"NULL" in L.moe_last_error()
        args[i] = ctypes.c_void_p(4100)
        assert call(L, name, args) == moe.MOE_ERR_INVALID_ARG, i
        assert b"aligned" in L.moe_last_error()
    assert call(L, name, [P] * n, desc=BAD) == moe.MOE_ERR_UNSUPPORTED
    assert call(L, name, [P] * n, desc=None) == moe.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("name", ["moe_expert_ffn_fwd_fp4", "moe_rms_norm_bwd"])
def test_small_workspace(L, name):
    assert call(L, name, [P] * CALLS[name][0], ws_bytes=8) == moe.MOE_ERR_INVALID_ARG
    assert b"workspace" in L.moe_last_error()


def test_rows_moved_in_sectors_are_32_byte_aligned(L):
    for i in (7, 8, 9, 11):
        args = [P] * 13
        args[i] = ctypes.c_void_p(4096 + 16)
        assert call(L, "moe_expert_ffn_fwd_fp4", args) == moe.MOE_ERR_INVALID_ARG, i
        assert b"32-byte aligned" in L.moe_last_error()


def test_values_of_both_weights_or_of_none(L):
    for i in (6, 7):
        args = [P] * 8
        args[i] = None
        assert call(L, "moe_fp4_quantize_weights", args) == moe.MOE_ERR_INVALID_ARG
        assert b"together" in L.moe_last_error()


@pytest.mark.parametrize("null,why", [((1,), b"r is the sum"), ((4, 5, 6), b"both NULL"),
                                      ((5,), b"together"), ((6,), b"together")])
def test_norm_outputs_that_do_not_go_together(L, null, why):
    args = [None if i in null else P for i in range(8)]
    assert call(L, "moe_rms_norm", args) == moe.MOE_ERR_INVALID_ARG
    assert why in L.moe_last_error()


@pytest.mark.parametrize("eps", [-1e-6, float("nan"), float("inf")])
def test_norm_eps(L, eps):
    assert call(L, "moe_rms_norm", [P] * 8, eps=eps) == moe.MOE_ERR_INVALID_ARG
    assert b"eps" in L.moe_last_error()


def test_scale_bytes(L):
    assert moe.moe_fp4_scale_bytes(10, 1) == 80 and moe.moe_fp4_scale_bytes(10, 8) == 80
    assert moe.moe_fp4_scale_bytes(9, 9) == 160 and moe.moe_fp4_scale_bytes(0, 5) == 0
    assert moe.moe_fp4_scale_bytes(1 << 31, 64) == 1 << 37  # past 32 bits
    assert moe.moe_fp4_scale_bytes(-1, 4) == 0 and moe.moe_fp4_scale_bytes(4, -1) == 0


def test_norm_workspace(L):
    size = lambda T, H: moe.moe_rms_norm_bwd_workspace_size(moe.LayerDesc.of(T, H, 1, 1, 64))  # noqa: E731
    assert size(0, 64) == 256 and size(10, 64) == 2560
    assert size(1 << 20, 2048) == size(1 << 24, 2048) > 0  # bounded
    with pytest.raises(moe.MoeError):
        moe.moe_rms_norm_bwd_workspace_size(BAD)


def bufs(**null):
    b, q = moe.MbBufs(), moe.Fp4Bufs()
    for n in moe._MB_FIELDS + moe._MB_FIELDS_TAIL:
        setattr(b, n, None if n in null else 4096)
    for n in moe._FP4_FIELDS:
        setattr(q, n, None if n in null else 4096)
    b.ws_bytes = moe.moe_workspace_size(D)
    return b, q


@pytest.mark.parametrize("missing", ["w1q", "w2s", "xq", "xs", "hq", "hs", "x", "slot", "o", "y",
                                     "x_perm", "a", "h", "ws"])
def test_layer_forward_needs(L, missing):
    b, q = bufs(**{missing: 1})
    st = L.moe_layer_forward_fp4(ctypes.byref(D), ctypes.byref(b), ctypes.byref(q), 1, None)
    assert st == moe.MOE_ERR_INVALID_ARG and b"NULL" in L.moe_last_error()


def test_layer_call_needs_its_structs(L):
    b, q = bufs()
    fn = L.moe_layer_forward_fp4
    assert fn(ctypes.byref(D), None, ctypes.byref(q), 1, None) == moe.MOE_ERR_INVALID_ARG
    assert fn(ctypes.byref(D), ctypes.byref(b), None, 1, None) == moe.MOE_ERR_INVALID_ARG
    assert fn(None, ctypes.byref(b), ctypes.byref(q), 1, None) == moe.MOE_ERR_INVALID_ARG


def test_binding_refuses_cpu_tensors():
    z = torch.zeros
    bf, u8 = torch.bfloat16, torch.uint8
    with pytest.raises(moe.MoeError, match="not on the current CUDA device"):
        moe.moe_rms_norm(D, z(16, 192, dtype=bf), None, z(192, dtype=bf), 1e-6, None,
                         z(16, 192, dtype=bf))
    with pytest.raises(moe.MoeError, match="x is torch.float32"):
        moe.moe_permute_fp4(D, z(16, 192), z(16, 2, dtype=torch.int32), z(32, 96, dtype=u8),
                            z(1, 32, 8, dtype=u8))
    with pytest.raises(moe.MoeError, match="dy is None"):
        moe.moe_rms_norm_bwd(D, None, None, None, None, None, None, None, None)


def test_buffers_of_other_layers_are_refused():
    other = moe.LayerDesc.of(T=16, H=192, E=8, k=2, F=256)
    with pytest.raises(moe.MoeError, match="another layer"):
        moe.Fp4Buffers(other, device="cpu", weights=moe.Fp4Buffers(D, device="cpu"))
    f = moe.Fp4Buffers(D, device="cpu")
    assert f.xs.numel() == moe.moe_fp4_scale_bytes(32, 6) and f.hs.shape == (1, 32, 8)
    b = moe.LayerBuffers(D, device="cpu")
    for d in (other, moe.LayerDesc.of(T=17, H=192, E=8, k=2, F=192),
              moe.LayerDesc.of(T=16, H=192, E=8, k=2, F=192, R=2)):
        with pytest.raises(moe.MoeError, match="another layer"):
            moe.moe_layer_forward_fp4(d, b, f)
    with pytest.raises(moe.MoeError, match="not on the current CUDA device"):
        moe.moe_layer_forward_fp4(D, b, f)
