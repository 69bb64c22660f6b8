"""fp32 weight gradients of many rows lose no more than their roundings (needs a
B200). The tensor cores cut their fp32 sums towards zero every 16 terms, on
average by half a unit in the last place, 0.36 * 2^-23 of the sum as it is then.
Over a part of 896 terms, 56 steps of a sum that is two thirds of the last one on
average, that is 1.6e-6; each further part adds one rounding, at most 2^-24 of
the whole. An unbroken sum of 8192 equal-signed terms loses 512 * 0.36 * 2^-23 / 2
= 1.1e-5 or more."""
import pytest
import torch

import test_gpu_train as T
from mixture_experts_layer_limited_b200 import native as N
from train_util import F32_U, F64

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def _bound(rows):
    return 1.6e-6 + (-(-rows // 896) + 4) * F32_U                # four more: each of up to four pairs rounds its last part up


# few tiles, split over four and over two pairs of SMs; as many as there are pairs, and more
@pytest.mark.parametrize("T_,H,E", [(8192, 256, 16), (8192, 7168, 256), (8191, 8960, 256), (6001, 8960, 208),
                                    (4097, 20480, 256)])
def test_fp32_gate_gradient_is_not_cut_short(T_, H, E):
    g = torch.Generator(device=DEV)
    g.manual_seed(T_ + H)
    dl, x = ((torch.rand(T_, n, generator=g, device=DEV) + 0.25).to(BF) for n in (E, H))
    ref = dl.to(F64).T @ x.to(F64)
    out = torch.empty(E, H, device=DEV)
    N.moe_gate_backward(T_, H, E, dl, x, None, None, None, out, grad_dtype=N.MOE_F32)
    assert float((out.to(F64) - ref).norm() / ref.norm()) < _bound(T_)
    again = torch.zeros_like(out)
    N.moe_gate_backward(T_, H, E, dl, x, None, None, None, again, grad_dtype=N.MOE_F32, accumulate=True)
    assert torch.equal(out, again)


@pytest.mark.parametrize("H,I", [(512, 384), (2048, 1408)])
def test_fp32_expert_gradients_are_not_cut_short(H, I):
    """8192 copies of one row: every row's part of a gradient is the same product
    of two bf16 numbers, which one row alone gives exactly."""
    R = 8192
    c, _, _, _ = T._case([1], H, I, seed=71)
    one = T._backward(c, None, 1, 1, H, I, f32=True, row_w=False, want=("d_w13", "d_w2"))
    many = {k: v.expand(R, *v.shape[1:]).contiguous() if k in ("a", "gu", "d_out", "row_w") else v for k, v in c.items()}
    got = T._backward(many, None, R, 1, H, I, f32=True, row_w=False, want=("d_w13", "d_w2"))
    for k in ("d_w13", "d_w2"):
        ref = R * one[k].to(F64)
        assert float((got[k].to(F64) - ref).norm() / ref.norm()) < _bound(R), k


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("counts,H,I", [([896, 897, 0, 2000, 911, 960, 961, 1, 1793, 4000], 512, 384),
                                        ([897], 256, 128), ([3600, 0, 1], 256, 256), ([4500], 2048, 1408)])
def test_fp32_gradients_of_segments_in_parts(counts, H, I, accumulate):
    """Segments of one, two and more parts, ending anywhere in a block of 64 rows,
    next to one another."""
    c, off, R, E = T._case(counts, H, I, seed=73)
    g = T._gen(74)
    init = [torch.randn(E, *n, generator=g, device=DEV) for n in ((2 * I, H), (H, I))] if accumulate else None
    o = T._backward(c, off, R, E, H, I, f32=True, accumulate=accumulate, init=init)
    again = T._backward(c, off, R, E, H, I, f32=True, accumulate=accumulate, init=init)
    for k, v in o.items():
        assert torch.equal(v, again[k])
    if accumulate:                               # one rounding of a sum of at most |init| + |gradient|
        ref, mag, fp = T.ffn_backward(c["a"], c["gu"], c["d_out"], c["w13"], c["w2"], off, c["row_w"])
        for k, i in zip(("d_w13", "d_w2"), init):
            tol = T.backward_tolerance(k, ref[k], mag[k], fp.get(k), H, I, max(counts), torch.float32)
            tol = tol + F32_U * (i.to(F64) + ref[k]).abs() * 2
            assert bool(((o[k].to(F64) - i.to(F64) - ref[k]).abs() <= tol).all()), k
    else:
        T._check(o, c, off, H, I)


def test_wait_limit_in_fp32_parts():
    """The wait limit in weight gradients that come in parts: the call gives up,
    flags it, and the same call with the default limit gives what it gave before."""
    H, I = 512, 384
    c, off, R, E = T._case([4000, 0, 1000], H, I, seed=79)
    before = T._backward(c, off, R, E, H, I, f32=True)
    offs = torch.tensor(off, dtype=torch.int32, device=DEV)
    ws = torch.empty(N.moe_swiglu_ffn_backward_workspace_size(R, I), dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    d13, d2 = torch.zeros_like(before["d_w13"]), torch.zeros_like(before["d_w2"])
    N.moe_set_wait_limit_ns(5)
    try:
        N.moe_swiglu_ffn_backward(R, H, c["w13"], c["w2"], E, I, c["a"], c["gu"], c["d_out"], offs, c["row_w"], None, d13, d2,
                                  None, ws, grad_dtype=N.MOE_F32, dev_status=status)
        assert N.moe_read_device_status(status) == N.MOE_DEVSTAT_TIMEOUT
    finally:
        N.moe_set_wait_limit_ns(0)
    after = T._backward(c, off, R, E, H, I, f32=True)
    for k in before:
        assert torch.equal(before[k], after[k])
