"""moe_route_backward's outputs over its inputs or one another (no GPU: every call
below is refused before any launch)."""
import ctypes
import os

import pytest

from mixture_experts_layer_limited_b200 import native as N
from mixture_experts_layer_limited_b200.build import lib_path

pytestmark = pytest.mark.skipif(not os.path.exists(lib_path()), reason="libmoe.so not built (run the package build)")
T, E, K = 64, 48, 6


def at(i, past=0):
    """An address of its own, never dereferenced."""
    return ctypes.c_void_p(0x10000000 * (i + 1) + past)


def test_overlapping_outputs_are_refused():
    """One warp a token: an output over another token's input, or over the other
    output, would be a race."""
    lib = N.load_library()

    def route(logits=at(0), ids=at(1), dw=at(2), s2r=at(3), out=at(4), out16=at(5)):
        return lib.moe_route_backward(T, E, K, N.MOE_SOFTMAX, 1, ctypes.c_float(1.0), logits, ids, dw, s2r, out, out16,
                                      None, None)
    for kw in (dict(out=at(0, 16)), dict(out=at(1)), dict(out=at(2)), dict(out=at(3, T * K * 4 - 16)), dict(out16=at(0)),
               dict(out16=at(1)), dict(out16=at(4)), dict(out16=at(4, T * E * 4 - 16)), dict(dw=at(5, T * E * 2 - 16)),
               dict(out=at(0), out16=at(0))):
        assert route(**kw) == N.MOE_ERR_INVALID_ARG, kw
    assert lib.moe_last_cuda_error() == 0
