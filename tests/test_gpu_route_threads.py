"""The router from two host threads at once (needs a B200)."""
import pytest
import torch

from mixture_experts_layer_limited_b200 import native as N
from test_gpu_threads import _at_once

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def test_gate_logits_of_different_expert_counts():
    """16 and 240 experts take different amounts of shared memory from the same
    kernel."""
    H, T = 256, 64
    lib = N.load_library()
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    calls, keep = [], []
    for E in (16, 240):
        x, gate = (torch.randn(n, H, generator=g, device=DEV).to(BF) for n in (T, E))
        out = torch.empty(T, E, device=DEV)
        args = (T, H, E, x.data_ptr(), gate.data_ptr(), out.data_ptr(), None)
        assert lib.moe_gate_logits(*args, None) == N.MOE_OK
        torch.cuda.synchronize()
        calls.append(args)
        keep.append((out, out.clone(), x, gate))
    assert not _at_once(lib.moe_gate_logits, calls)
    for out, want, _, _ in keep:
        assert torch.equal(out, want)
