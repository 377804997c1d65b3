"""The 8-bit experts' host-side checks (no GPU work): the C entry points and the
binding refuse bad arguments before anything is launched."""
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
    "moe_fp8_quantize_weights": (6, ()),
    "moe_permute_fp8": (4, ()),
    "moe_expert_ffn_fwd_fp8": (13, (7, 8)),
    "moe_combine_bwd_fp8": (8, (4,)),
    "moe_expert_ffn_bwd_dgrad_fp8": (13, (8,)),
}


def call(L, name, args, desc=D, ws_bytes=None):
    tail = ()
    if CALLS[name][0] == 13:
        tail = (moe.moe_workspace_size(D) if ws_bytes is None else ws_bytes,)
    return getattr(L, name)(ctypes.byref(desc), *args, *tail, None)


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
    assert getattr(L, name)(None, *[P] * n, *([0] if n == 13 else []), None) == moe.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("name", ["moe_expert_ffn_fwd_fp8", "moe_expert_ffn_bwd_dgrad_fp8"])
def test_small_workspace(L, name):
    assert call(L, name, [P] * 13, ws_bytes=8) == moe.MOE_ERR_INVALID_ARG
    assert b"workspace" in L.moe_last_error()


@pytest.mark.parametrize("name,at", [("moe_expert_ffn_fwd_fp8", (7, 8, 9, 11)),
                                     ("moe_expert_ffn_bwd_dgrad_fp8", (2, 8, 9, 11))])
def test_rows_moved_in_sectors_are_32_byte_aligned(L, name, at):
    for i in at:
        args = [P] * 13
        args[i] = ctypes.c_void_p(4096 + 16)
        assert call(L, name, args) == moe.MOE_ERR_INVALID_ARG, i
        assert b"32-byte aligned" in L.moe_last_error()


def test_scale_bytes(L):
    assert moe.moe_fp8_scale_bytes(10, 1) == 40 and moe.moe_fp8_scale_bytes(10, 4) == 40
    assert moe.moe_fp8_scale_bytes(10, 5) == 80 and moe.moe_fp8_scale_bytes(0, 5) == 0
    assert moe.moe_fp8_scale_bytes(1 << 31, 128) == 1 << 38  # past 32 bits
    assert moe.moe_fp8_scale_bytes(-1, 4) == 0 and moe.moe_fp8_scale_bytes(4, -1) == 0


def bufs(**null):
    b, q = moe.MbBufs(), moe.Fp8Bufs()
    for n in moe._MB_FIELDS + moe._MB_FIELDS_TAIL:
        setattr(b, n, None if n in null else 4096)
    for n in moe._FP8_FIELDS:
        setattr(q, n, None if n in null else 4096)
    b.ws_bytes = moe.moe_workspace_size(D)
    return b, q


@pytest.mark.parametrize("missing", ["w1q", "w2s", "xq", "xs", "hq", "hs", "x", "slot", "o", "y",
                                     "x_perm", "a", "h", "ws"])
def test_layer_forward_needs(L, missing):
    b, q = bufs(**{missing: 1})
    st = L.moe_layer_forward_fp8(ctypes.byref(D), ctypes.byref(b), ctypes.byref(q), 1, None)
    assert st == moe.MOE_ERR_INVALID_ARG and b"NULL" in L.moe_last_error()


@pytest.mark.parametrize("missing", ["w1q", "dq", "ds", "daq", "das", "dy", "a", "o", "dx",
                                     "x_perm", "h", "d_o", "da", "dw1"])
def test_layer_backward_needs(L, missing):
    b, q = bufs(**{missing: 1})
    st = L.moe_layer_backward_fp8(ctypes.byref(D), ctypes.byref(b), ctypes.byref(q), 1, None)
    assert st == moe.MOE_ERR_INVALID_ARG and b"NULL" in L.moe_last_error()


def test_layer_calls_need_their_structs(L):
    b, q = bufs()
    for fn in (L.moe_layer_forward_fp8, L.moe_layer_backward_fp8):
        assert fn(ctypes.byref(D), None, ctypes.byref(q), 1, None) == moe.MOE_ERR_INVALID_ARG
        assert fn(ctypes.byref(D), ctypes.byref(b), None, 1, None) == moe.MOE_ERR_INVALID_ARG
        assert fn(None, ctypes.byref(b), ctypes.byref(q), 1, None) == moe.MOE_ERR_INVALID_ARG


def test_binding_refuses_wrong_tensors(L):
    """Types, places, shapes and strides, on the CPU: nothing here could be launched."""
    x = torch.zeros(16, 192, dtype=torch.bfloat16)
    slot = torch.zeros(16, 2, dtype=torch.int32)
    xq = torch.zeros(32, 192, dtype=torch.uint8).view(torch.float8_e4m3fn)
    xs = torch.zeros(1, 32, 4, dtype=torch.uint8)
    with pytest.raises(moe.MoeError, match="CUDA device"):
        moe.moe_permute_fp8(D, x, slot, xq, xs, stream=0)
    with pytest.raises(moe.MoeError, match="float32"):
        moe.moe_permute_fp8(D, x.float(), slot, xq, xs, stream=0)
    with pytest.raises(moe.MoeError, match="x is None"):
        moe.moe_permute_fp8(D, None, slot, xq, xs, stream=0)


@pytest.mark.gpu
def test_binding_refuses_strided_and_small_tensors(L):
    x = torch.zeros(16, 192, dtype=torch.bfloat16, device="cuda")
    slot = torch.zeros(16, 2, dtype=torch.int32, device="cuda")
    xq = torch.zeros(32, 192, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    xs = torch.zeros(1, 32, 4, dtype=torch.uint8, device="cuda")
    with pytest.raises(moe.MoeError, match="uint8"):
        moe.moe_permute_fp8(D, x, slot, xq.view(torch.uint8), xs)
    with pytest.raises(moe.MoeError, match="contiguous"):
        moe.moe_permute_fp8(D, torch.zeros(192, 16, dtype=torch.bfloat16, device="cuda").t(), slot,
                            xq, xs)
    with pytest.raises(moe.MoeError, match="elements"):
        moe.moe_permute_fp8(D, x[:15], slot, xq, xs)
    with pytest.raises(moe.MoeError, match="elements"):
        moe.moe_permute_fp8(D, x, slot, xq, xs[:, :31])
    with pytest.raises(moe.MoeError, match="aligned"):
        big = torch.zeros(16 * 192 + 1, dtype=torch.bfloat16, device="cuda")
        moe.moe_permute_fp8(D, big[1:].view(16, 192), slot, xq, xs)


@pytest.mark.parametrize("call", ["moe_layer_forward_fp8", "moe_layer_backward_fp8"])
@pytest.mark.parametrize("other", [dict(T=15), dict(H=128), dict(E=4), dict(k=1), dict(F=128)])
def test_layer_calls_refuse_buffers_of_another_layer(call, other):
    small = moe.LayerDesc.of(**{**dict(T=16, H=192, E=8, k=2, F=192), **other})
    mine = moe.LayerBuffers(D, "cpu"), moe.Fp8Buffers(D, "cpu")
    theirs = moe.LayerBuffers(small, "cpu"), moe.Fp8Buffers(small, "cpu")
    for b, q, name in ((theirs[0], mine[1], "bufs"), (mine[0], theirs[1], "fp8")):
        with pytest.raises(moe.MoeError, match=f"{name} is of another layer"):
            getattr(moe, call)(D, b, q)


def test_buffer_struct_follows_the_tensors():
    q = moe.Fp8Buffers(D, "cpu")
    before = q.struct().w1q
    q.w1q = torch.empty_like(q.w1q)
    assert q.struct().w1q == q.w1q.data_ptr() != before


@pytest.mark.parametrize("call", ["moe_layer_forward_fp8", "moe_layer_backward_fp8"])
def test_layer_calls_refuse_buffers_in_host_memory(call):
    with pytest.raises(moe.MoeError, match="CUDA device"):
        getattr(moe, call)(D, moe.LayerBuffers(D, "cpu"), moe.Fp8Buffers(D, "cpu"))


@pytest.mark.parametrize("other", [dict(H=128), dict(E=4), dict(F=128)])
def test_shared_weights_are_of_the_same_layer(other):
    q = moe.Fp8Buffers(D, "cpu")
    assert moe.Fp8Buffers(moe.LayerDesc.of(T=1, H=192, E=8, k=1, F=192), "cpu", weights=q).w1q is q.w1q
    theirs = moe.LayerDesc.of(**{**dict(T=16, H=192, E=8, k=2, F=192), **other})
    with pytest.raises(moe.MoeError, match="another layer"):
        moe.Fp8Buffers(theirs, "cpu", weights=q)


@pytest.mark.parametrize("call", ["moe_layer_forward_fp8", "moe_layer_backward_fp8"])
@pytest.mark.parametrize("mine,theirs", [(8, 1), (1, 8), (2, 4)])
def test_layer_calls_refuse_buffers_of_another_number_of_ranks(call, mine, theirs):
    """rank_off has R + 1 entries, which the layout writes: R=1's buffers are too small for R=8."""
    of = lambda r: moe.LayerDesc.of(T=16, H=192, E=8, k=2, F=192, R=r)  # noqa: E731
    with pytest.raises(moe.MoeError, match=f"bufs is of another layer: .*R={theirs}$"):
        getattr(moe, call)(of(mine), moe.LayerBuffers(of(theirs), "cpu"), moe.Fp8Buffers(of(mine), "cpu"))
    # the 8-bit buffers do not depend on it: the call gets as far as their place
    with pytest.raises(moe.MoeError, match="CUDA device"):
        getattr(moe, call)(of(mine), moe.LayerBuffers(of(mine), "cpu"), moe.Fp8Buffers(of(theirs), "cpu"))


@pytest.mark.parametrize("call", ["moe_layer_forward_fp8", "moe_layer_backward_fp8"])
def test_buffers_know_the_sizes_that_they_were_made_for(call):
    """A descriptor changed after its buffers were made does not take them along."""
    d = moe.LayerDesc.of(T=16, H=192, E=8, k=2, F=192)
    b, q = moe.LayerBuffers(d, "cpu"), moe.Fp8Buffers(d, "cpu")
    d.T = 32
    with pytest.raises(moe.MoeError, match="bufs is of another layer: T=16 "):
        getattr(moe, call)(d, b, q)
    with pytest.raises(moe.MoeError, match="fp8 is of another layer: T=16 "):
        getattr(moe, call)(d, moe.LayerBuffers(d, "cpu"), q)


def test_scale_bytes_of_the_largest_counts(L):
    most = (1 << 31) - 1
    assert moe.moe_fp8_scale_bytes(1, most) == 1 << 31
    assert moe.moe_fp8_scale_bytes(3, most - 3) == 3 * (most - 3)
