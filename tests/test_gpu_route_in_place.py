"""moe_route_backward writing d_logits over the logits (needs a B200)."""
import pytest
import torch

from mixture_experts_layer_limited_b200 import native as N

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("scoring", [N.MOE_SOFTMAX, N.MOE_SIGMOID])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("T,E,k", [(1, 16, 4), (513, 64, 6), (2000, 256, 16)])
def test_in_place_of_the_logits(scoring, norm, T, E, k):
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    logits = torch.randn(T, E, generator=g, device=DEV) * 2
    ids = torch.rand(T, E, generator=g, device=DEV).topk(k, dim=1)[1].to(torch.int32)
    dw = torch.randn(T, k, generator=g, device=DEV)
    out, out16, got16 = torch.empty_like(logits), *(torch.empty(T, E, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    N.moe_route_backward(T, E, k, scoring, norm, 2.5, logits, ids, dw, None, out, out16)
    N.moe_route_backward(T, E, k, scoring, norm, 2.5, logits, ids, dw, None, logits, got16)
    assert torch.equal(logits, out) and torch.equal(got16, out16)
