"""Outputs over memory that every kernel of a chain reads (no GPU: every call
below is refused before any launch)."""
import ctypes
import os

import pytest

from mixture_experts_layer_limited_b200 import native as N
from mixture_experts_layer_limited_b200.build import lib_path

pytestmark = pytest.mark.skipif(not os.path.exists(lib_path()), reason="libmoe.so not built (run the package build)")
E, H, I, R = 4, 512, 256, 64


def at(i, past=0):
    """An address of its own, never dereferenced."""
    return ctypes.c_void_p(0x10000000 * (i + 1) + past)


def _w():
    w = N.FFNWeights(at(0), at(1), None, None, N.MOE_BF16, E, I)
    w.tiled = 0
    return w


def test_outputs_over_the_offsets_are_refused():
    lib, w = N.load_library(), _w()

    def train(h=at(3), gu=at(4), off=at(5)):
        return lib.moe_gate_up_swiglu_train(R, H, ctypes.byref(w), at(2), off, h, gu, None, None)
    assert train(h=at(5)) == N.MOE_ERR_INVALID_ARG
    assert train(gu=at(5, 16)) == N.MOE_ERR_INVALID_ARG                   # the last of E + 1 = 5 words
    assert train(off=at(4, R * I * 4 - 16)) == N.MOE_ERR_INVALID_ARG

    need = N.moe_swiglu_ffn_backward_workspace_size(R, I)

    def back(d_a=at(6), d13=at(7), d2=at(8), drw=at(9), ws=at(10), off=at(5)):
        return lib.moe_swiglu_ffn_backward(R, H, ctypes.byref(w), at(2), at(4), at(3), off, at(11), d_a, d13, d2,
                                           N.MOE_BF16, 0, drw, ws, need, None, None)
    for kw in (dict(d_a=at(5)), dict(d13=at(5)), dict(d2=at(5, 16)), dict(drw=at(5)), dict(ws=at(5)),
               dict(off=at(10, need - 16)), dict(off=at(9, R * 4 - 16))):
        assert back(**kw) == N.MOE_ERR_INVALID_ARG, kw
    assert lib.moe_last_cuda_error() == 0
