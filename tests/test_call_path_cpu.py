"""What the checked call path refuses before it looks at any tensor (CPU)."""
import ctypes

import pytest
import torch

import combine_router_softmax_top_gb300 as moe

BF, U8, I32 = torch.bfloat16, torch.uint8, torch.int32


class Lookalike(ctypes.Structure):
    """Has a descriptor's sizes by name, but not its layout: the library would read past it."""
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "H", "E", "k", "F")]


class NoCtypes:
    T, H, E, k, F = 4, 64, 2, 1, 64


def calls(d):
    z = lambda *s, dt=BF: torch.zeros(*s, dtype=dt)  # noqa: E731
    x, w1, w2 = z(4, 64), z(2, 128, 64), z(2, 64, 64)
    b = z(1 << 16, dt=U8)
    yield lambda: moe.moe_permute_fp4(d, x, z(4, dt=I32), b, b)
    yield lambda: moe.moe_fp4_quantize_weights(d, w1, w2, b, b, b, b)
    yield lambda: moe.moe_expert_ffn_fwd_fp4(d, b, b, z(3, dt=I32), b, b, b, b, None, None, b, b, x, b)
    yield lambda: moe.moe_rms_norm(d, x, None, z(64), 1e-6, None, x)
    yield lambda: moe.moe_rms_norm_bwd(d, x, None, x, z(64), z(4, dt=torch.float32), x,
                                       z(64, dt=torch.float32), b)
    yield lambda: moe.moe_permute_fp8(d, x, z(4, dt=I32), z(4, 64, dt=torch.float8_e4m3fn), b)


@pytest.mark.parametrize("desc", [Lookalike(4, 64, 2, 1, 64), NoCtypes()])
def test_another_descriptor(desc):
    """As every other call of the library: a descriptor is a LayerDesc."""
    for call in calls(desc):
        with pytest.raises(ctypes.ArgumentError, match="LayerDesc"):
            call()
    with pytest.raises(ctypes.ArgumentError):
        moe.lib().moe_workspace_size(ctypes.byref(desc) if isinstance(desc, ctypes.Structure) else desc)


def test_a_descriptor_of_a_derived_class_is_one():
    class Mine(moe.LayerDesc):
        pass
    d = moe.LayerDesc.of(4, 64, 2, 1, 64)
    mine = Mine.from_buffer_copy(bytes(d))
    for call in calls(mine):
        with pytest.raises(moe.MoeError, match="device"):  # (the next thing that is wrong here)
            call()
