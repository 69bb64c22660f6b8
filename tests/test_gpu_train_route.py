"""moe_route_backward where the chosen experts' scores leave fp32's range (needs a
B200): renormalised weights are ratios of scores, finite however small the
scores are."""
import pytest
import torch

from mixture_experts_layer_limited_b200 import native as N
from train_util import F32_U, F64, route_weights

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("shift", [-60.0, -87.0, -89.0, -95.0, -120.0, 40.0])
def test_renormalised_weights_of_tiny_scores(scoring, shift):
    """Chosen logits around `shift`, others up to zero; one token with a chosen
    logit of -inf, which has no share and no gradient."""
    T, E, k = 65, 64, 6
    g = torch.Generator(device=DEV)
    g.manual_seed(int(200 + shift))
    logits = torch.randn(T, E, generator=g, device=DEV) * 2
    ids = torch.rand(T, E, generator=g, device=DEV).topk(k, dim=1)[1]
    logits.scatter_(1, ids, torch.randn(T, k, generator=g, device=DEV) * 3 + shift)
    logits[7, ids[7, 2]] = float("-inf")
    dw = torch.randn(T, k, generator=g, device=DEV)
    # ratios of scores as softmax over the chosen: of the logits, or of log sigmoid
    x = logits.to(F64).requires_grad_()
    chosen = x.gather(1, ids)
    z = chosen if scoring == "softmax" else torch.nn.functional.logsigmoid(chosen)
    r = torch.softmax(z, 1)
    ref, = torch.autograd.grad((2.5 * r * dw.to(F64)).sum(), x)
    ref = ref.nan_to_num()                                                # the -inf logit's own (0 * inf in the formula)
    if shift == -60.0:                                                    # the same weights as the definition's, there in range
        fin = torch.isfinite(logits).all(1)
        assert torch.allclose(2.5 * r[fin], route_weights(x.detach(), ids, scoring, True, 2.5)[fin], rtol=1e-9)
    out = torch.full((T, E), 7.0, device=DEV)
    code = N.MOE_SOFTMAX if scoring == "softmax" else N.MOE_SIGMOID
    N.moe_route_backward(T, E, k, code, True, 2.5, logits, ids.to(torch.int32), dw, None, out)
    # 64 roundings of the terms, as where scores are ordinary; the exponent's argument, a difference of up to 40, is
    # rounded once: 40 roundings of its exponential
    share = torch.zeros(T, E, dtype=F64, device=DEV).scatter(1, ids, r.detach())
    most = 2.5 * (dw.abs().to(F64) + (dw.abs() * r.detach()).sum(1, keepdim=True)).amax(1, keepdim=True)
    err = (out.to(F64) - ref).abs()
    assert bool((err <= (64 + 40) * F32_U * most * share * k + 1e-30).all()), float(err.max())
