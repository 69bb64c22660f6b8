"""The first CUDA call of a host thread is one of the library's (needs a B200)."""
import threading

import pytest
import torch

from mixture_experts_layer_limited_b200 import native as N

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
H, I, R, E = 256, 128, 40, 16


def _call(name):
    """(call, outputs) of an entry point that takes tensor maps."""
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV).to(BF)
    x, gate, w13, w2, gu, d_out = n(R, H), n(E, H), n(1, 2 * I, H), n(1, H, I), n(R, 2 * I), n(R, H)
    new = lambda *s, dtype=BF: torch.zeros(*s, dtype=dtype, device=DEV)
    if name == "gate logits":
        o = [new(R, E, dtype=torch.float32)]
        return lambda: N.moe_gate_logits(R, H, E, x, gate, *o), o
    if name == "experts":
        o = [new(R, I), new(R, H)]
        return lambda: N.moe_grouped_swiglu(R, H, w13, w2, N.MOE_BF16, 1, I, x, None, None, *o), o
    if name == "4-bit experts":
        code = lambda *s: torch.randint(0, 256, s, generator=g, device=DEV, dtype=torch.uint8)
        scale = lambda *s: torch.full(s, 120, dtype=torch.uint8, device=DEV)
        q13, q2, a = code(1, 2 * I, H // 2), code(1, H, I // 2), code(R, H // 2)
        s = dict(w13_scale=scale(1, 2 * I // 128, H // 128, 512), w2_scale=scale(1, H // 128, I // 128, 512),
                 a_scale=scale(H // 128, R, 4))
        o = [new(R, I // 2, dtype=torch.uint8), new(R, H), new(I // 128, R, 4, dtype=torch.uint8)]
        return lambda: N.moe_grouped_swiglu(R, H, q13, q2, N.MOE_MXFP4, 1, I, a, None, None, o[0], o[1], h_scale_ws=o[2], **s), o
    if name == "training forward":
        o = [new(R, I), new(R, 2 * I)]
        return lambda: N.moe_gate_up_swiglu_train(R, H, w13, 1, I, x, None, *o), o
    if name == "backward":
        o = [new(R, H), new(1, 2 * I, H), new(1, H, I), new(R, dtype=torch.float32)]
        ws = new(N.moe_swiglu_ffn_backward_workspace_size(R, I), dtype=torch.uint8)
        return lambda: N.moe_swiglu_ffn_backward(R, H, w13, w2, 1, I, x, gu, d_out, None, None, *o, ws), o
    o = [new(R, H), new(E, H)]
    dl = n(R, E)
    return lambda: N.moe_gate_backward(R, H, E, dl, x, gate, None, *o), o


@pytest.mark.parametrize("name", ["gate logits", "experts", "4-bit experts", "training forward", "backward", "gate backward"])
def test_first_call_of_a_thread(name):
    call, outs = _call(name)
    call()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    raised = []

    def work():
        try:
            call()
        except Exception as e:               # handed to the test
            raised.append(e)
    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not raised
    for o, w in zip(outs, want):
        assert torch.equal(o, w)
