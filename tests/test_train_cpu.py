"""Host-side checks of the training and 4-bit entry points, and the float64
formulas of their tests against differences (no GPU: every call below is
refused before any launch)."""
import ctypes
import os

import pytest
import torch

from mixture_experts_layer_limited_b200 import native as N
from mixture_experts_layer_limited_b200.build import lib_path
import mx_util as X
from train_util import F64, ffn_backward, ffn_forward, route_weights

built = pytest.mark.skipif(not os.path.exists(lib_path()), reason="libmoe.so not built (run the package build)")
P = ctypes.c_void_p
FAKE, ODD = P(0x1000), P(0x1004)          # never dereferenced


def _w(dtype=N.MOE_BF16, groups=4, I=256, tiled=0, w13=FAKE, w2=FAKE, scale=None):
    w = N.FFNWeights(w13, w2, scale, scale, dtype, groups, I)
    w.tiled = tiled
    return w


@built
def test_train_forward_refusals():
    lib = N.load_library()

    def call(w, rows=8, H=512, a=FAKE, off=FAKE, h=FAKE, gu=FAKE):
        return lib.moe_gate_up_swiglu_train(rows, H, ctypes.byref(w), a, off, h, gu, None, None)
    assert call(_w(), rows=0) == N.MOE_ERR_INVALID_ARG
    assert call(_w(), gu=None) == N.MOE_ERR_INVALID_ARG
    assert call(_w(), off=None) == N.MOE_ERR_INVALID_ARG                 # one group only without offsets
    assert call(_w(), H=384) == N.MOE_ERR_UNSUPPORTED
    assert call(_w(I=192)) == N.MOE_ERR_UNSUPPORTED
    assert call(_w(), gu=ODD) == N.MOE_ERR_ALIGNMENT
    assert call(_w(dtype=N.MOE_E4M3, scale=FAKE)) != N.MOE_OK
    assert call(_w(dtype=N.MOE_MXFP4, scale=FAKE)) != N.MOE_OK
    assert lib.moe_last_cuda_error() == 0


@built
def test_backward_refusals():
    lib = N.load_library()
    rows, I = 64, 256
    need = N.moe_swiglu_ffn_backward_workspace_size(rows, I)
    assert need == rows * (6 * I + 4 * (I // 32))
    with pytest.raises(N.MoEError):
        N.moe_swiglu_ffn_backward_workspace_size(0, I)
    with pytest.raises(N.MoEError):
        N.moe_swiglu_ffn_backward_workspace_size(rows, 100)

    def call(w=None, H=512, a=FAKE, gu=FAKE, d_out=FAKE, off=FAKE, d_a=FAKE, d13=FAKE, d2=FAKE, dt=N.MOE_BF16, acc=0,
             drw=FAKE, ws=FAKE, nbytes=need, r=rows):
        w = w if w is not None else _w()
        return lib.moe_swiglu_ffn_backward(r, H, ctypes.byref(w), a, gu, d_out, off, FAKE, d_a, d13, d2, dt, acc, drw, ws,
                                           nbytes, None, None)
    assert call(nbytes=need - 1) == N.MOE_ERR_INVALID_ARG
    assert call(ws=None) == N.MOE_ERR_INVALID_ARG
    assert call(gu=None) == N.MOE_ERR_INVALID_ARG
    assert call(d_out=None) == N.MOE_ERR_INVALID_ARG
    assert call(a=None) == N.MOE_ERR_INVALID_ARG                          # d_w13 needs the rows
    assert call(_w(w13=None)) == N.MOE_ERR_INVALID_ARG                    # d_a needs w13
    assert call(d_a=None, d13=None, d2=None, drw=None) == N.MOE_ERR_INVALID_ARG
    assert call(off=None) == N.MOE_ERR_INVALID_ARG
    assert call(dt=N.MOE_E4M3) == N.MOE_ERR_INVALID_ARG
    assert call(acc=1) == N.MOE_ERR_INVALID_ARG                           # bf16 gradients do not accumulate
    assert call(acc=2, dt=N.MOE_F32) == N.MOE_ERR_INVALID_ARG
    assert call(ws=ODD) == N.MOE_ERR_ALIGNMENT
    assert call(d13=ODD) == N.MOE_ERR_ALIGNMENT
    assert call(H=200) == N.MOE_ERR_UNSUPPORTED
    assert call(_w(groups=513)) == N.MOE_ERR_UNSUPPORTED
    assert call(_w(dtype=N.MOE_MXFP4, scale=FAKE)) != N.MOE_OK
    assert lib.moe_last_cuda_error() == 0


@built
def test_router_and_gate_backward_refusals():
    lib = N.load_library()

    def route(T=8, E=64, k=4, scoring=N.MOE_SOFTMAX, logits=FAKE, ids=FAKE, dw=FAKE, out=FAKE, out16=FAKE):
        return lib.moe_route_backward(T, E, k, scoring, 0, ctypes.c_float(1.0), logits, ids, dw, None, out, out16, None, None)
    assert route(T=0) == N.MOE_ERR_INVALID_ARG
    assert route(k=65) == N.MOE_ERR_INVALID_ARG
    assert route(scoring=2) == N.MOE_ERR_INVALID_ARG
    assert route(dw=None) == N.MOE_ERR_INVALID_ARG
    assert route(E=24) == N.MOE_ERR_UNSUPPORTED
    assert route(E=512) == N.MOE_ERR_UNSUPPORTED
    assert route(k=17) == N.MOE_ERR_UNSUPPORTED
    assert route(out16=ODD) == N.MOE_ERR_ALIGNMENT

    def gate(T=8, H=512, E=64, dl=FAKE, x=FAKE, g=FAKE, dx_in=FAKE, dx=FAKE, dg=FAKE, dt=N.MOE_BF16, acc=0):
        return lib.moe_gate_backward(T, H, E, dl, x, g, dx_in, dx, dg, dt, acc, None, None)
    assert gate(T=0) == N.MOE_ERR_INVALID_ARG
    assert gate(dl=None) == N.MOE_ERR_INVALID_ARG
    assert gate(dx=None, dx_in=None, dg=None) == N.MOE_ERR_INVALID_ARG
    assert gate(dx=None) == N.MOE_ERR_INVALID_ARG                         # dx_in without dx
    assert gate(g=None) == N.MOE_ERR_INVALID_ARG
    assert gate(x=None) == N.MOE_ERR_INVALID_ARG
    assert gate(acc=1) == N.MOE_ERR_INVALID_ARG
    assert gate(dt=7) == N.MOE_ERR_INVALID_ARG
    assert gate(H=384) == N.MOE_ERR_UNSUPPORTED
    assert gate(E=40) == N.MOE_ERR_UNSUPPORTED
    assert gate(dg=ODD) == N.MOE_ERR_ALIGNMENT
    assert lib.moe_last_cuda_error() == 0


@built
def test_mxfp4_refusals():
    lib = N.load_library()

    def rows(r=8, K=256, a=FAKE, a_rows=8, src=None, q=FAKE, s=FAKE):
        return lib.moe_quantize_mxfp4_rows(r, K, a, a_rows, src, q, s, None, None)
    assert rows(r=0) == N.MOE_ERR_INVALID_ARG
    assert rows(a_rows=7) == N.MOE_ERR_INVALID_ARG                        # fewer source rows and no map
    assert rows(s=None) == N.MOE_ERR_INVALID_ARG
    assert rows(K=160) == N.MOE_ERR_UNSUPPORTED
    assert rows(q=ODD) == N.MOE_ERR_ALIGNMENT
    assert lib.moe_dequantize_mxfp4_rows(8, 100, FAKE, FAKE, FAKE, None) == N.MOE_ERR_UNSUPPORTED
    assert lib.moe_dequantize_mxfp4_rows(8, 128, FAKE, None, FAKE, None) == N.MOE_ERR_INVALID_ARG
    assert lib.moe_quantize_mxfp4_weights(1, 100, 128, FAKE, FAKE, FAKE, None) == N.MOE_ERR_UNSUPPORTED
    assert lib.moe_quantize_mxfp4_weights(1, 128, 128, FAKE, FAKE, ODD, None) == N.MOE_ERR_ALIGNMENT

    def ffn(w, a_scale=FAKE, h_scale=FAKE, H=512):
        return lib.moe_grouped_swiglu(8, H, ctypes.byref(w), FAKE, a_scale, FAKE, None, FAKE, h_scale, FAKE, None, None)
    mx = lambda **kw: _w(dtype=N.MOE_MXFP4, scale=kw.pop("scale", FAKE), **kw)
    assert ffn(mx(scale=None)) == N.MOE_ERR_INVALID_ARG
    assert ffn(mx(), a_scale=None) == N.MOE_ERR_INVALID_ARG
    assert ffn(mx(), h_scale=None) == N.MOE_ERR_INVALID_ARG
    assert ffn(mx(tiled=1)) == N.MOE_ERR_UNSUPPORTED
    assert ffn(mx(I=192)) == N.MOE_ERR_UNSUPPORTED
    assert ffn(mx(), H=384) == N.MOE_ERR_UNSUPPORTED
    assert ffn(mx(), a_scale=ODD) == N.MOE_ERR_ALIGNMENT
    assert lib.moe_last_cuda_error() == 0


@built
def test_overlapping_outputs_are_refused():
    """The products of a call run beside one another, so an output in an input's
    or another output's memory would be read after being written."""
    lib = N.load_library()
    at = lambda i: P(0x10000000 * (i + 1))                                # far apart; never dereferenced
    E, H, I, R = 4, 512, 256, 64
    w = _w(w13=at(0), w2=at(1))

    def train(a=at(2), h=at(3), gu=at(4)):
        return lib.moe_gate_up_swiglu_train(R, H, ctypes.byref(w), a, at(5), h, gu, None, None)
    assert train(h=at(2)) == N.MOE_ERR_INVALID_ARG
    assert train(gu=P(at(3).value + R * I * 2 - 16)) == N.MOE_ERR_INVALID_ARG

    need = N.moe_swiglu_ffn_backward_workspace_size(R, I)

    def back(d_a=at(6), d13=at(7), d2=at(8), drw=at(9), ws=at(10)):
        return lib.moe_swiglu_ffn_backward(R, H, ctypes.byref(w), at(2), at(4), at(3), at(5), at(11), d_a, d13, d2,
                                           N.MOE_BF16, 0, drw, ws, need, None, None)
    for kw in (dict(d_a=at(2)), dict(d_a=at(3)), dict(d13=at(0)), dict(d2=at(7)), dict(drw=at(11)), dict(ws=at(4)),
               dict(d_a=P(at(3).value + R * H * 2 - 16)), dict(drw=P(at(10).value + need - 16))):
        assert back(**kw) == N.MOE_ERR_INVALID_ARG, kw

    def gate(x=at(12), dx_in=at(13), dx=at(14), dg=at(15)):
        return lib.moe_gate_backward(R, H, 64, at(16), x, at(17), dx_in, dx, dg, N.MOE_BF16, 0, None, None)
    assert gate(dx=at(12)) == N.MOE_ERR_INVALID_ARG
    assert gate(dx_in=P(at(14).value + 16)) == N.MOE_ERR_INVALID_ARG      # dx itself, or apart from it
    assert gate(dg=at(17)) == N.MOE_ERR_INVALID_ARG
    assert lib.moe_quantize_mxfp4_rows(8, 256, at(0), 8, at(1), at(0), at(2), None, None) == N.MOE_ERR_INVALID_ARG
    assert lib.moe_quantize_mxfp4_rows(8, 256, at(0), 8, at(1), at(2), at(2), None, None) == N.MOE_ERR_INVALID_ARG
    assert lib.moe_dequantize_mxfp4_rows(8, 256, at(0), at(1), at(0), None) == N.MOE_ERR_INVALID_ARG
    assert lib.moe_quantize_mxfp4_weights(1, 128, 256, at(0), at(0), at(1), None) == N.MOE_ERR_INVALID_ARG
    assert lib.moe_last_cuda_error() == 0


# ------------------------------------------------- the tests' own formulas
def test_backward_formula_against_differences():
    """The float64 formula of the GPU tests: every gradient along random
    directions against central differences (error of order eps^2)."""
    torch.manual_seed(1)
    off = [1, 4, 4, 9]
    R, E, H, I = 10, 3, 16, 8
    n = lambda *s: torch.randn(*s, dtype=F64)
    a, w13, w2, row_w, d_out = n(R, H), n(E, 2 * I, H) * 0.3, n(E, H, I) * 0.3, torch.rand(R, dtype=F64) + 0.1, n(R, H)
    gu = ffn_forward(a, w13, w2, off, row_w)[0]
    g, _, _ = ffn_backward(a, gu, d_out, w13, w2, off, row_w)
    args = dict(a=a, w13=w13, w2=w2, row_w=row_w)
    eps = 1e-6
    for gname, name in dict(d_a="a", d_w13="w13", d_w2="w2", d_row_w="row_w").items():
        for _ in range(3):
            d = torch.randn_like(args[name])
            f = [(ffn_forward(**{**args, name: args[name] + s * eps * d}, offsets=off)[2] * d_out).sum() for s in (1, -1)]
            assert float((g[gname] * d).sum()) == pytest.approx(float((f[0] - f[1]) / (2 * eps)), rel=1e-6, abs=1e-7)


@pytest.mark.parametrize("scoring,norm", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
def test_route_formula_against_differences(scoring, norm):
    torch.manual_seed(2)
    x = torch.randn(5, 16, dtype=F64, requires_grad=True)
    ids = torch.stack([torch.randperm(16)[:4] for _ in range(5)])
    dw = torch.randn(5, 4, dtype=F64)
    f = lambda v: (route_weights(v, ids, scoring, norm, 2.5) * dw).sum()
    g, = torch.autograd.grad(f(x), x)
    d, eps = torch.randn_like(x), 1e-6
    diff = (f(x + eps * d) - f(x - eps * d)) / (2 * eps)
    assert float((g * d).sum()) == pytest.approx(float(diff.detach()), rel=1e-6, abs=1e-8)


def test_mx_definition_on_known_blocks():
    """Codes and scales worked out by hand: amax 6 -> scale 1; ties at 0.25,
    0.75, 1.25, 1.75, 2.5, 3.5, 5 go to the even code; 7 saturates to 6."""
    v = torch.zeros(1, 32)
    v[0, :10] = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -7.0, -0.0])
    code, s = X.quantize(v)
    assert s.tolist() == [[127]]
    assert code[0, :10].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 15, 8]
    assert X.values(code, s)[0, :9].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, -6]
    assert X.scale_bytes(torch.full((1, 32), 4.0)).item() == 127 and X.scale_bytes(torch.full((1, 32), 3.99)).item() == 126
    assert X.scale_bytes(torch.zeros(1, 32)).item() == 127
    assert X.scale_bytes(torch.full((1, 32), float("nan"))).item() == 255
    assert torch.equal(X.unpack(X.pack(code)), code)
