"""A training step of the whole layer, and the 4-bit layer's forward, against
float64 (needs a B200). The choice of experts is taken from the layer; all else
is recomputed.

Gradients are compared in the 2-norm: each passes at most six bf16 roundings
one after the other (pre-activations, h, o, d_o's rows, dg/du, d_xp, the result),
each relative error at most U_bf16 on its values: 7 U_bf16 of the norm."""
import dataclasses

import pytest
import torch

import mx_util as X
from mixture_experts_layer_limited_b200 import LayerSpec, MoELayer
from moe_inputs import get_config, make_inputs, tiny_grouped_config
from train_util import BF16_U, F64, route_weights

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _cfg(name):
    return {"tiny": get_config("tiny"), "grouped": tiny_grouped_config(),
            "noshared": dataclasses.replace(get_config("tiny"), I_s=0),
            "wide": dataclasses.replace(tiny_grouped_config(), H=768, I=384, I_s=640, T=200, k=6, E=32)}[name]


def _layer(cfg, **kw):
    inp = make_inputs(cfg, device=DEV)
    shared = (inp.sw13, inp.sw2) if cfg.I_s else (None, None)
    return inp, MoELayer(LayerSpec.from_config(cfg), inp.gate, inp.w13, inp.w2, *shared, inp.bias, cfg.T, **kw)


def _reference(cfg, inp, ids, x, gate, w13, w2, sw13=None, sw2=None):
    """y of the layer for the given expert ids, differentiable, float64."""
    w = route_weights(x @ gate.T, ids, cfg.scoring, cfg.norm_topk_prob, cfg.scale)
    ffn = lambda v, a, b: (torch.nn.functional.silu(v @ a.T[:, :a.shape[0] // 2]) * (v @ a.T[:, a.shape[0] // 2:])) @ b.T
    y = torch.zeros_like(x)
    for e in range(cfg.E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if len(t):
            y = y.index_add(0, t, w[t, j, None] * ffn(x[t], w13[e], w2[e]))
    return y if sw13 is None else y + ffn(x, sw13, sw2)


def _norm_err(got, ref):
    return float((got.to(F64) - ref).norm() / ref.norm())


@pytest.mark.parametrize("tiled", [True, False])
@pytest.mark.parametrize("name", ["tiny", "grouped", "noshared", "wide"])
def test_training_step(name, tiled):
    cfg = _cfg(name)
    inp, layer = _layer(cfg, tiled_weights=tiled)
    T = cfg.T - 1                                        # a batch smaller than the layer's buffers
    x, g = inp.x[:T].contiguous(), torch.Generator(device=DEV)
    g.manual_seed(5)
    dy = (torch.randn(T, cfg.H, generator=g, device=DEV) * 0.1).to(torch.bfloat16)
    y = layer.forward_train(x).clone()
    assert torch.equal(y, layer.forward(x))              # the inference forward's y
    layer.forward_train(x)
    grads = layer.grad_buffers()
    dx = layer.backward(dy, grads)
    assert layer.device_status() == 0
    leaves = {"x": x, "gate": inp.gate, "w13": inp.w13, "w2": inp.w2}
    if cfg.I_s:
        leaves.update(sw13=inp.sw13, sw2=inp.sw2)
    leaves = {k: v.to(F64).requires_grad_() for k, v in leaves.items()}
    ref_y = _reference(cfg, inp, layer.ids[:T].long(), **leaves)
    assert _norm_err(y, ref_y.detach()) <= 7 * BF16_U
    refs = dict(zip(leaves, torch.autograd.grad((ref_y * dy.to(F64)).sum(), list(leaves.values()))))
    for k, ref in refs.items():
        got = dx if k == "x" else grads[k]
        assert _norm_err(got.reshape(ref.shape), ref) <= 7 * BF16_U, k


def test_training_step_accumulates_in_fp32():
    cfg = _cfg("grouped")
    inp, layer = _layer(cfg)
    dy = torch.ones_like(inp.x) * 0.1
    layer.forward_train(inp.x)
    once = layer.grad_buffers(torch.float32)
    layer.backward(dy, once)
    twice = layer.grad_buffers(torch.float32)
    for _ in range(2):
        layer.forward_train(inp.x)
        layer.backward(dy, twice, accumulate=True)
    for k in once:
        assert torch.equal(twice[k], 2 * once[k])        # equal addends: exact


def test_training_step_captured_and_replayed():
    """The step as one CUDA graph, replayed on other inputs, gives the eager
    step's gradients bit for bit."""
    cfg = _cfg("wide")
    inp, layer = _layer(cfg)
    x, dy = inp.x.clone(), (inp.x * 0.1).contiguous()
    grads = layer.grad_buffers()

    def step():
        layer.forward_train(x)
        return layer.backward(dy, grads)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dx = step()
    for scale in (1.0, -0.5):
        x.copy_(inp.x * scale)
        dy.copy_(inp.x * 0.2 * scale)
        graph.replay()
        got = {k: v.clone() for k, v in grads.items()}
        got["x"] = dx.clone()
        for v in grads.values():
            v.zero_()
        got_eager = step()
        assert torch.equal(got.pop("x"), got_eager)
        for k, v in got.items():
            assert torch.equal(v, grads[k]), k


def test_training_refusals():
    cfg = _cfg("tiny")
    inp, layer = _layer(cfg)
    with pytest.raises(ValueError):
        layer.backward(inp.x, layer.grad_buffers())      # no forward_train
    layer.forward_train(inp.x)
    layer.forward(inp.x)
    with pytest.raises(ValueError):
        layer.backward(inp.x, layer.grad_buffers())      # a forward() took its buffers
    layer.forward_train(inp.x)
    with pytest.raises(ValueError):
        layer.backward(inp.x[:3], layer.grad_buffers())
    with pytest.raises(ValueError):
        layer.backward(inp.x, {"w13": layer.grad_buffers()["w13"]})
    with pytest.raises(ValueError):
        layer.forward_train(layer.forward(inp.x))        # its own output buffer, overwritten before backward()
    inp4, layer4 = _layer(dataclasses.replace(cfg, dtype="mxfp4"))
    with pytest.raises(ValueError):
        layer4.forward_train(inp4.x)


# ------------------------------------------------------------------ 4 bits
@pytest.mark.parametrize("name", ["tiny", "grouped", "noshared", "wide"])
def test_mxfp4_layer(name):
    """The 4-bit layer against float64 with the same quantisation. h's codes may
    step to a neighbour where h lies between two: rare (its fp32 error against
    a step of a quarter), so the 2-norm is held to bf16's roundings of o and y
    and one such step (a third of a value) in a thousand values."""
    cfg = dataclasses.replace(_cfg(name), dtype="mxfp4")
    inp, layer = _layer(cfg)
    T = cfg.T - 3
    x = inp.x[:T].contiguous()
    y = layer.forward(x).clone()
    assert layer.device_status() == 0
    qdq = lambda v: X.values(*X.quantize(v))
    xq = qdq(x)
    ids, w = layer.ids[:T].long(), layer.topk_w[:T].to(F64)

    def ffn(v, a, b):
        a, b = qdq(a), qdq(b)
        I = a.shape[0] // 2
        gu = v @ a.T
        return qdq(torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]) @ b.T
    ref = ffn(xq, inp.sw13, inp.sw2) if cfg.I_s else torch.zeros(T, cfg.H, dtype=F64, device=DEV)
    for e in range(cfg.E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if len(t):
            ref.index_add_(0, t, w[t, j, None] * ffn(xq[t], inp.w13[e], inp.w2[e]))
    assert _norm_err(y, ref) <= 2 * BF16_U + 0.34 * 1e-3 ** 0.5
    again = layer.forward(x)
    assert torch.equal(y, again)


def test_mxfp4_layer_through_the_host_pipeline():
    from mixture_experts_layer_limited_b200 import HostPipeline
    cfg = dataclasses.replace(_cfg("wide"), dtype="mxfp4")
    inp, layer = _layer(cfg)
    xs = [(inp.x * s).cpu().pin_memory() for s in (1.0, -2.0, 0.5)]
    want = [layer.forward(x.to(DEV)).cpu().clone() for x in xs]
    ys = [torch.empty_like(x).pin_memory() for x in xs]
    HostPipeline(layer, cfg.T).run(xs, ys)
    torch.cuda.synchronize()
    for y, w in zip(ys, want):
        assert torch.equal(y, w)


def test_mxfp4_layer_captured():
    cfg = dataclasses.replace(_cfg("wide"), dtype="mxfp4")
    inp, layer = _layer(cfg)
    y = layer.forward(inp.x).clone()
    replay = layer.capture(inp.x)
    layer.y.zero_()
    replay()
    assert torch.equal(layer.y[:cfg.T], y)
