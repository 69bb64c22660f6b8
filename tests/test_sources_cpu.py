"""Rules of the kernel sources that no result shows (no GPU)."""
import os
import re

import pytest

from mixture_experts_layer_limited_b200.build import CSRC

# kernels launched with programmatic stream serialization, and what they share
EARLY = ["train.cu", "mxfp4.cu", "segments.cuh"]


def _kernels(text):
    """Bodies of a file's kernels, by name."""
    attributes = r"(?:__\w+__\s*\((?:[^()]|\([^()]*\))*\)\s*)*"
    starts = list(re.finditer(r"__global__\s+void\s+" + attributes + r"(\w+)\s*\([^;{]*\)\s*\{", text))
    ends = [m.start() for m in starts[1:]] + [len(text)]
    return {m.group(1): text[m.start():e] for m, e in zip(starts, ends)}


@pytest.mark.parametrize("name", EARLY)
def test_kernels_that_start_early_load_plainly(name):
    """A kernel that starts while the one before it still writes must not read
    that one's results through the read-only path, whose data the compiler may
    take to be constant for the whole kernel."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    assert "__ldg" not in text and "ld.global.nc" not in text
    for kernel, body in _kernels(text).items():
        if "griddep_wait()" in body:
            assert "__restrict__" not in body.split("{", 1)[0], kernel


def test_the_rule_sees_the_kernels():
    with open(os.path.join(CSRC, "mxfp4.cu")) as f:
        found = _kernels(f.read())
    assert {"mx_quant_rows_kernel", "mx_dequant_rows_kernel", "mx_gemm_kernel"} <= set(found)
    assert "griddep_wait()" in found["mx_gemm_kernel"] and "griddep_wait()" not in found["mx_quant_weights_kernel"]
