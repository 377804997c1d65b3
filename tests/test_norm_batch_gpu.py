"""What a token's norm depends on beside the token (include/moe.h, moe_rms_norm): for H <= 2048
nothing, above that also on whether there are more tokens than multiprocessors."""
import pytest
import torch

import combine_router_softmax_top_gb300 as moe

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    from combine_router_softmax_top_gb300 import build
    build.build()


def norm(x, res, w):
    T, H = x.shape
    d = moe.LayerDesc.of(T, H, 1, 1, 64)
    r, y = torch.empty_like(x), torch.empty_like(x)
    yq = torch.zeros(T, H, device="cuda").to(torch.float8_e4m3fn)
    ys = torch.zeros(-(-H // 512), T, 4, dtype=torch.uint8, device="cuda")
    rstd = torch.empty(T, device="cuda")
    moe.moe_rms_norm(d, x, res, w, 1e-6, r, y, yq, ys, rstd)
    return r, y, yq.view(torch.uint8), ys.transpose(0, 1).contiguous(), rstd


@pytest.mark.parametrize("H", [64, 128, 320, 576, 1024, 2048, 2112, 4096, 16384])
def test_a_tokens_bits(H):
    g = torch.Generator(device="cuda").manual_seed(H)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    x, res = ((torch.randn(2 * sms + 3, H, generator=g, device="cuda") * s).to(BF) for s in (1.0, 3.0))
    w = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(BF)
    few = [norm(x[:n].contiguous(), res[:n].contiguous(), w) for n in (1, 2, 7, sms)]
    many = [norm(x[:n].contiguous(), res[:n].contiguous(), w) for n in (sms + 1, 2 * sms + 3)]
    for group in ([few + many] if H <= 2048 else [few, many]):
        for out in group:
            n = out[4].numel()
            for got, want in zip(out, group[-1]):
                m = min(n, want.shape[0])
                assert torch.equal(got[:m], want[:m])
    # on both sides the sums, over H squares in another order, are within their error
    a, b = few[-1][4].double(), many[0][4][:sms].double()
    assert ((a - b).abs() <= (H + 16) * 2.0 ** -24 * a).all()
