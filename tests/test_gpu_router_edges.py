"""GPU tests of moe_router_logits' workspace."""
import pytest
import torch

from mixture_experts_ffn_topk_amd import MoEError, MoEFFN

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)


def test_bf16_weights_need_no_workspace():
    """At a size where fp32 weights need one and are refused without it."""
    T, H, E = 4100, 1024, 256
    g = torch.Generator().manual_seed(1)
    x = torch.randn(T, H, generator=g).bfloat16().cuda()
    w = (torch.randn(E, H, generator=g) * H ** -0.5).cuda()
    moe = MoEFFN(H, 64, E, 1, T, fmt="w4a8_mx")
    assert moe.router_workspace_size(T) > 0
    with_ws, without = torch.empty(T, E, device="cuda"), torch.empty(T, E, device="cuda")
    moe.router_logits(T, x, w.bfloat16(), with_ws, moe.alloc_router_workspace(T))
    moe.router_logits(T, x, w.bfloat16(), without)
    assert torch.equal(with_ws, without)
    with pytest.raises(MoEError, match="WORKSPACE_TOO_SMALL"):
        moe.router_logits(T, x, w, without)
