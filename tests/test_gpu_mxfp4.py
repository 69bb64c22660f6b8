"""MXFP4 quantisers and experts' products of libmoe against the format's
definition in float64 (needs a B200). Codes and scales bit for bit; products of
codes are exact, so only fp32 sums and the output's rounding remain."""
import pytest
import torch

import mx_util as X
from mixture_experts_layer_limited_b200 import native as N
from train_util import BF16_U, F32_U, F64, segments

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _rows(R, K, seed):
    """Rows over the whole range of scales, with ties, zeros and saturation."""
    g = _gen(seed)
    x = torch.randn(R, K, generator=g, device=DEV)
    x = x * torch.exp2(torch.randint(-30, 31, (R, 1), generator=g, device=DEV).float())
    x[::5] = torch.randint(-28, 29, (x[::5].shape), generator=g, device=DEV) / 4      # quarters: every tie
    return x.to(BF)


def _quant(x, src=None, rows=None):
    rows = rows if rows is not None else (src.numel() if src is not None else x.shape[0])
    K = x.shape[1]
    q = torch.full((rows, K // 2), 0xAA, dtype=torch.uint8, device=DEV)
    s = torch.full((K // 128, rows, 4), 0xAA, dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    N.moe_quantize_mxfp4_rows(rows, K, x, x.shape[0], src, q, s, dev_status=status)
    return q, s, N.moe_read_device_status(status)


@pytest.mark.parametrize("R,K", [(1, 128), (7, 256), (33, 1408), (65, 2048), (3, 7168), (130, 640)])
def test_quantize_rows_bytes(R, K):
    x = _rows(R, K, R + K)
    q, s, st = _quant(x)
    code, scale = X.quantize(x)
    assert st == 0
    assert torch.equal(s, X.row_scale_words(scale))
    assert torch.equal(q, X.pack(code))
    out = torch.empty(R, K, dtype=BF, device=DEV)
    N.moe_dequantize_mxfp4_rows(R, K, q, s, out)
    assert torch.equal(out.to(F64), X.values(code, scale))


def test_quantize_rows_gathered():
    x = _rows(9, 384, 1)
    src = torch.tensor([8, 0, 0, 3, 8, 5, 1, 2, 2, 2, 7], dtype=torch.int32, device=DEV)
    q, s, st = _quant(x, src)
    code, scale = X.quantize(x[src.long()])
    assert st == 0 and torch.equal(q, X.pack(code)) and torch.equal(s, X.row_scale_words(scale))
    bad = src.clone()
    bad[2], bad[5] = 9, -1
    q2, s2, st = _quant(x, bad)
    assert st & N.MOE_DEVSTAT_BAD_EXPERT_ID
    assert bool((q2[[2, 5]] == 0).all()) and bool((s2[:, [2, 5]] == 127).all())
    keep = [0, 1, 3, 4, 6, 7, 8, 9, 10]
    assert torch.equal(q2[keep], q[keep]) and torch.equal(s2[:, keep], s[:, keep])


def test_quantize_extremes():
    """Blocks of zeros, of the smallest and largest numbers, of a lone outlier,
    and with NaN or infinity (scale 255: the block's values are NaN)."""
    x = torch.zeros(8, 128, dtype=BF, device=DEV)
    x[1, 5] = -0.0
    x[2, :32] = 2.0 ** -133                                   # the smallest subnormal
    x[3, :32] = torch.finfo(BF).max
    x[4, 7] = -1e30
    x[4, 8] = 1.0
    x[5, 40] = float("nan")
    x[6, 70] = float("-inf")
    x[7, :] = torch.finfo(BF).tiny
    q, s, st = _quant(x)
    code, scale = X.quantize(x)
    assert st == 0 and torch.equal(s, X.row_scale_words(scale))
    finite = (scale != 255).repeat_interleave(32, 1)
    assert torch.equal(X.unpack(q)[finite], code[finite])
    out = torch.empty(8, 128, dtype=BF, device=DEV)
    N.moe_dequantize_mxfp4_rows(8, 128, q, s, out)
    assert bool(torch.isnan(out[5, 32:64]).all()) and bool(torch.isnan(out[6, 64:96]).all())
    assert torch.equal(out.to(F64)[finite], X.values(code, scale)[finite])


@pytest.mark.parametrize("B,Nr,K", [(1, 128, 128), (3, 256, 384), (2, 384, 1408)])
def test_quantize_weights_bytes(B, Nr, K):
    w = _rows(B * Nr, K, 5).reshape(B, Nr, K)
    q = torch.empty(B, Nr, K // 2, dtype=torch.uint8, device=DEV)
    s = torch.empty(B, Nr // 128, K // 128, 512, dtype=torch.uint8, device=DEV)
    N.moe_quantize_mxfp4_weights(B, Nr, K, w, q, s)
    code, scale = X.quantize(w)
    assert torch.equal(q, X.pack(code)) and torch.equal(s, X.weight_scale_blocks(scale))


def _layer(counts, H, I, seed, lead=0, behind=0):
    g = _gen(seed)
    off = segments(counts, lead)
    E, R = len(counts), off[-1] + behind
    n = lambda *s, std=1.0: torch.randn(*s, generator=g, device=DEV) * std
    w13c, w13s = X.quantize(n(E, 2 * I, H, std=0.05))
    w2c, w2s = X.quantize(n(E, H, I, std=0.05))
    # rows of widely different scales, so that a scale taken from a neighbour shows
    xc, xs = X.quantize(n(R, H) * torch.exp2(torch.randint(-2, 3, (R, H // 32), generator=g, device=DEV).float())
                        .repeat_interleave(32, 1))
    hc, hs = X.quantize(n(R, I) * torch.exp2(torch.randint(-3, 4, (R, I // 32), generator=g, device=DEV).float())
                        .repeat_interleave(32, 1))
    row_w = torch.rand(R, generator=g, device=DEV) + 0.1
    return dict(w13=w13c, w13s=w13s, w2=w2c, w2s=w2s, x=xc, xs=xs, h=hc, hs=hs, row_w=row_w), off, R, E


SHAPES = [
    # counts, H, I: rows around the 16-, 32- and 64-row tiles, empty experts; K of an odd number of 128-blocks
    ([1], 256, 128),
    ([5, 0, 16, 1, 17], 512, 384),
    ([33, 31, 0, 64], 256, 256),
    ([70, 129, 3], 768, 640),
    ([200, 193, 257], 512, 1408),
    ([500, 0, 0, 2], 256, 128),
]


@pytest.mark.parametrize("counts,H,I", SHAPES)
def test_down_product(counts, H, I):
    c, off, R, E = _layer(counts, H, I, seed=H + I, lead=1, behind=2)
    out = torch.full((R, H), 7.0, dtype=BF, device=DEV)
    offs = torch.tensor(off, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    N.moe_down_proj(R, H, X.pack(c["w2"]), N.MOE_MXFP4, E, I, X.pack(c["h"]), offs, c["row_w"], out,
                    w2_scale=X.weight_scale_blocks(c["w2s"]), h_scale=X.row_scale_words(c["hs"]), dev_status=status)
    assert N.moe_read_device_status(status) == 0
    lo, hi = off[0], off[-1]
    assert bool((out[:lo] == 7).all()) and bool((out[hi:] == 7).all())
    h = X.values(c["h"], c["hs"])
    for e in range(E):
        s = slice(off[e], off[e + 1])
        w2 = X.values(c["w2"][e], c["w2s"][e])
        rw = c["row_w"][s].to(F64)[:, None]
        ref, mag = rw * (h[s] @ w2.T), rw * (h[s].abs() @ w2.abs().T)
        err = (out[s].to(F64) - ref).abs()
        assert bool((err <= BF16_U * ref.abs() * 1.01 + (I + 2) * F32_U * mag).all()), (e, float(err.max()))


@pytest.mark.parametrize("counts,H,I", SHAPES)
def test_gate_up_product(counts, H, I):
    """h's scales are the definition's where the block's largest value is clear
    of a power of two, and every code's value is as near to h as its grid allows."""
    c, off, R, E = _layer(counts, H, I, seed=H * 3 + I, lead=1, behind=2)
    q = torch.full((R, I // 2), 0x33, dtype=torch.uint8, device=DEV)
    s = torch.full((I // 128, R, 4), 0x33, dtype=torch.uint8, device=DEV)
    offs = torch.tensor(off, dtype=torch.int32, device=DEV)
    N.moe_gate_up_swiglu(R, H, X.pack(c["w13"]), N.MOE_MXFP4, E, I, X.pack(c["x"]), offs, q,
                         w13_scale=X.weight_scale_blocks(c["w13s"]), a_scale=X.row_scale_words(c["xs"]), h_scale_ws=s)
    lo, hi = off[0], off[-1]
    for a, b in ((0, lo), (hi, R)):
        assert bool((q[a:b] == 0x33).all()) and bool((s[:, a:b] == 0x33).all())
    x = X.values(c["x"], c["xs"])
    got_s = s.transpose(0, 1).reshape(R, -1).long()
    got = X.values(X.unpack(q), got_s)
    for e in range(E):
        r = slice(off[e], off[e + 1])
        if off[e] == off[e + 1]:
            continue
        w = X.values(c["w13"][e], c["w13s"][e])
        gu, mag = x[r] @ w.T, x[r].abs() @ w.abs().T
        g, u = gu[:, :I], gu[:, I:]
        h = g * torch.sigmoid(g) * u
        dg, du = H * F32_U * mag[:, :I], H * F32_U * mag[:, I:]
        # |silu'| <= 1.1, silu's own error 2^-20 (exp, fast division)
        tol = 1.1 * dg * u.abs() + g.abs() * du + 1.1 * dg * du + 2.0 ** -20 * h.abs()
        amax, atol = (t.reshape(t.shape[0], -1, 32).amax(-1) for t in (h.abs(), tol))
        lo_s, hi_s = (X.scale_bytes((amax + k * atol).clamp(min=0).repeat_interleave(32, 1)) for k in (-1, 1))
        assert bool(((got_s[r] >= lo_s) & (got_s[r] <= hi_s) | (amax <= atol)).all())
        unit = X.pow2(got_s[r] - 127).repeat_interleave(32, 1)
        near = (got[r] - h).abs() <= X.half_step((h.abs() + tol) / unit) * unit + tol
        assert bool(near.all())


def test_grouped_swiglu_and_shared():
    """Both products in one call, and with a shared expert, are the single calls'."""
    H, I, T = 512, 384, 20
    c, off, R, E = _layer([9, 0, 40, 11], H, I, seed=3)
    d, _, _, _ = _layer([T], H, 256, seed=4)
    offs = torch.tensor(off, dtype=torch.int32, device=DEV)
    u8 = dict(dtype=torch.uint8, device=DEV)
    pw = {k: X.pack(v[k]) for v in (c,) for k in ("w13", "w2", "x")}
    sw = {k: X.weight_scale_blocks(c[k]) for k in ("w13s", "w2s")}
    xs = X.row_scale_words(c["xs"])
    h, hs, out = torch.empty(R, I // 2, **u8), torch.empty(I // 128, R, 4, **u8), torch.empty(R, H, dtype=BF, device=DEV)
    N.moe_grouped_swiglu(R, H, pw["w13"], pw["w2"], N.MOE_MXFP4, E, I, pw["x"], offs, c["row_w"], h, out,
                         w13_scale=sw["w13s"], w2_scale=sw["w2s"], a_scale=xs, h_scale_ws=hs)
    hv = X.values(X.unpack(h), hs.transpose(0, 1).reshape(R, -1).long())
    for e in range(E):
        s = slice(off[e], off[e + 1])
        w2 = X.values(c["w2"][e], c["w2s"][e])
        rw = c["row_w"][s].to(F64)[:, None]
        ref, mag = rw * (hv[s] @ w2.T), rw * (hv[s].abs() @ w2.abs().T)
        assert bool(((out[s].to(F64) - ref).abs() <= BF16_U * ref.abs() * 1.01 + (I + 2) * F32_U * mag).all())
    h2, hs2, out2 = torch.empty_like(h), torch.empty_like(hs), torch.empty_like(out)
    sh, shs, so = torch.empty(T, 128, **u8), torch.empty(2, T, 4, **u8), torch.empty(T, H, dtype=BF, device=DEV)
    ref_sh, ref_shs, ref_so = torch.empty_like(sh), torch.empty_like(shs), torch.empty_like(so)
    pd = {k: X.pack(d[k]) for k in ("w13", "w2", "x")}
    sd = {k: X.weight_scale_blocks(d[k]) for k in ("w13s", "w2s")}
    dxs = X.row_scale_words(d["xs"])
    N.moe_gate_up_swiglu_with_shared(R, H, pw["w13"], N.MOE_MXFP4, E, I, pw["x"], offs, h2, T, pd["w13"], 256, pd["x"], sh,
                                     w13_scale=sw["w13s"], a_scale=xs, h_scale_ws=hs2, sw13_scale=sd["w13s"],
                                     sh_a_scale=dxs, sh_h_scale_ws=shs)
    N.moe_down_proj_with_shared(R, H, pw["w2"], N.MOE_MXFP4, E, I, h2, offs, c["row_w"], out2, T, pd["w2"], 256, sh, so,
                                w2_scale=sw["w2s"], h_scale=hs2, sw2_scale=sd["w2s"], sh_h_scale=shs)
    N.moe_grouped_swiglu(T, H, pd["w13"], pd["w2"], N.MOE_MXFP4, 1, 256, pd["x"], None, None, ref_sh, ref_so,
                         w13_scale=sd["w13s"], w2_scale=sd["w2s"], a_scale=dxs, h_scale_ws=ref_shs)
    assert torch.equal(h, h2) and torch.equal(hs, hs2) and torch.equal(out, out2)
    assert torch.equal(sh, ref_sh) and torch.equal(shs, ref_shs) and torch.equal(so, ref_so)


def test_nan_scale_stays_in_its_row():
    """A row with NaN gives NaN in its own output and nowhere else."""
    H, I = 256, 128
    c, off, R, E = _layer([20], H, I, seed=6)
    hs = c["hs"].clone()
    hs[7, 2] = 255
    out = torch.empty(R, H, dtype=BF, device=DEV)
    N.moe_down_proj(R, H, X.pack(c["w2"]), N.MOE_MXFP4, E, I, X.pack(c["h"]), None, None, out,
                    w2_scale=X.weight_scale_blocks(c["w2s"]), h_scale=X.row_scale_words(hs))
    assert bool(torch.isnan(out[7]).all()) and bool(torch.isfinite(out[:7]).all()) and bool(torch.isfinite(out[8:]).all())


def test_wait_limit_runs_out_then_the_same_call_is_correct():
    """As for the bf16 products: a wait limit of a few nanoseconds ends the
    kernels with MOE_DEVSTAT_TIMEOUT, and the same call is right afterwards."""
    H, I = 768, 384
    c, off, R, E = _layer([40, 0, 150, 3], H, I, seed=8)
    offs = torch.tensor(off, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    u8 = dict(dtype=torch.uint8, device=DEV)
    a, w13, w2 = X.pack(c["x"]), X.pack(c["w13"]), X.pack(c["w2"])
    s = dict(w13_scale=X.weight_scale_blocks(c["w13s"]), w2_scale=X.weight_scale_blocks(c["w2s"]),
             a_scale=X.row_scale_words(c["xs"]))

    def run():
        h, hs, out = torch.zeros(R, I // 2, **u8), torch.zeros(I // 128, R, 4, **u8), torch.zeros(R, H, dtype=BF, device=DEV)
        N.moe_grouped_swiglu(R, H, w13, w2, N.MOE_MXFP4, E, I, a, offs, c["row_w"], h, out, h_scale_ws=hs,
                             dev_status=status, **s)
        return (h, hs, out), N.moe_read_device_status(status)
    before, st = run()
    assert st == 0
    N.moe_set_wait_limit_ns(5)
    try:
        _, st = run()
    finally:
        N.moe_set_wait_limit_ns(0)
    assert st == N.MOE_DEVSTAT_TIMEOUT
    status.zero_()
    after, st = run()
    assert st == 0
    for x, y in zip(before, after):
        assert torch.equal(x, y)
