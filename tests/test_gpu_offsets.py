"""Forward products given offsets that do not describe segments of the rows
(needs a B200): segments are cut to the rows and to what lies behind the ones
before them, the call is flagged, and nothing outside the rows is touched. Every
product shares one schedule of tiles."""
import pytest
import torch

import mx_util as X
from mixture_experts_layer_limited_b200 import native as N

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
E, H, I, R, PAST = 4, 512, 384, 700, 1500

# given offsets, and the segments they are cut to
BAD = [([0, 300, 5000, 5000, 6000], [0, 300, 700, 700, 700]),       # past the rows
       ([-90, 20, 310, 500, 700], [0, 20, 310, 500, 700]),           # before them
       ([0, 600, 40, 650, 700], [0, 600, 600, 650, 700]),            # falling: behind what came before
       ([0, 2 ** 31 - 1, -2 ** 31, 650, 100], [0, 700, 700, 700, 700]),
       ([900, 1000, 1100, 1200, 1300], [700, 700, 700, 700, 700])]
CALLS = ["gate_up", "down", "grouped", "with_shared", "ffn", "down_combine", "gather", "e4m3", "mxfp4"]


def _inputs():
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=g, device=DEV) * std).to(BF)
    return dict(a=n(R, H), w13=n(E, 2 * I, H, std=0.05), w2=n(E, H, I, std=0.05), h=n(R, I), sw13=n(1, 2 * I, H, std=0.05),
                sw2=n(1, H, I, std=0.05), x=n(64, H), row_w=torch.rand(R, generator=g, device=DEV) + 0.1,
                tok=torch.randint(0, 64, (R,), generator=g, device=DEV, dtype=torch.int32))


def _run(call, c, off):
    """Outputs of the call (each with PAST rows behind it) and the device status."""
    offs = torch.tensor(off, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    big = lambda rows, cols, dtype=BF: torch.full((rows + PAST, cols), 7, dtype=dtype, device=DEV)
    h, out = big(R, I), big(R, H)
    kw = dict(dev_status=status)
    if call == "gate_up":
        N.moe_gate_up_swiglu(R, H, c["w13"], N.MOE_BF16, E, I, c["a"], offs, h[:R], **kw)
        got = [h]
    elif call == "down":
        N.moe_down_proj(R, H, c["w2"], N.MOE_BF16, E, I, c["h"], offs, c["row_w"], out[:R], **kw)
        got = [out]
    elif call == "grouped":
        N.moe_grouped_swiglu(R, H, c["w13"], c["w2"], N.MOE_BF16, E, I, c["a"], offs, c["row_w"], h[:R], out[:R], **kw)
        got = [h, out]
    elif call == "with_shared":
        sh, so = big(64, I), big(64, H)
        N.moe_gate_up_swiglu_with_shared(R, H, c["w13"], N.MOE_BF16, E, I, c["a"], offs, h[:R], 64, c["sw13"], I, c["x"],
                                         sh[:64], **kw)
        N.moe_down_proj_with_shared(R, H, c["w2"], N.MOE_BF16, E, I, h[:R], offs, c["row_w"], out[:R], 64, c["sw2"], I,
                                    sh[:64], so[:64], **kw)
        got = [h, out, sh, so]
    elif call == "ffn":
        sh, so = big(64, I), big(64, H)
        sync = torch.zeros(N.moe_swiglu_ffn_sync_size(R, E, 64) // 4 + 4096, dtype=torch.int32, device=DEV)
        N.moe_swiglu_ffn_with_shared(R, H, c["w13"], c["w2"], E, I, c["a"], offs, c["row_w"], h[:R], out[:R], 64, c["sw13"],
                                     c["sw2"], I, c["x"], sh[:64], so[:64], sync[:-4096], **kw)
        assert not bool(sync[-4096:].any())
        got = [h, out, sh, so]
    elif call == "down_combine":
        acc = big(64, H, torch.float32)
        acc[:64] = 0
        y = big(64, H)
        N.moe_down_proj_combine(R, 64, H, c["w2"], E, I, c["h"], offs, c["row_w"], c["tok"], None, 0, None, acc[:64],
                                y[:64], **kw)
        got = [y]
    elif call == "gather":
        N.moe_gate_up_swiglu_gather(R, H, c["w13"], E, I, c["x"], 64, c["tok"], offs, h[:R], **kw)
        got = [h]
    elif call == "e4m3":
        (w13, s13), (w2, s2) = _blocks(c["w13"]), _blocks(c["w2"])
        a, sa = torch.empty(R, H, dtype=torch.uint8, device=DEV), torch.empty(R, H // 128, device=DEV)
        N.moe_quantize_rows(R, H, c["a"], a, sa)
        h, hs = big(R, I, torch.uint8), big(R, I // 128, torch.float32)
        N.moe_grouped_swiglu(R, H, w13, w2, N.MOE_E4M3, E, I, a, offs, c["row_w"], h[:R], out[:R], w13_scale=s13, w2_scale=s2,
                             a_scale=sa, h_scale_ws=hs[:R], **kw)
        got = [h, hs, out]
    else:
        (w13, s13), (w2, s2) = _mx(c["w13"]), _mx(c["w2"])
        code, s = X.quantize(c["a"])
        h, hs = big(R, I // 2, torch.uint8), torch.full((I // 128, R, 4), 7, dtype=torch.uint8, device=DEV)
        N.moe_grouped_swiglu(R, H, w13, w2, N.MOE_MXFP4, E, I, X.pack(code), offs, c["row_w"], h[:R], out[:R], w13_scale=s13,
                             w2_scale=s2, a_scale=X.row_scale_words(s), h_scale_ws=hs, **kw)
        got = [h, out]
    return got, N.moe_read_device_status(status)


def _blocks(w):
    q = torch.empty(w.shape, dtype=torch.uint8, device=DEV)
    s = torch.empty(w.shape[0], w.shape[1] // 128, w.shape[2] // 128, device=DEV)
    N.moe_quantize_blocks(*w.shape, w, q, s)
    return q, s


def _mx(w):
    B, n, k = w.shape
    q = torch.empty(B, n, k // 2, dtype=torch.uint8, device=DEV)
    s = torch.empty(B, n // 128, k // 128, 512, dtype=torch.uint8, device=DEV)
    N.moe_quantize_mxfp4_weights(B, n, k, w, q, s)
    return q, s


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("given,cut", BAD)
def test_bad_offsets_are_cut_and_flagged(call, given, cut):
    c = _inputs()
    got, status = _run(call, c, given)
    want, clean = _run(call, c, cut)
    assert status == N.MOE_DEVSTAT_BAD_EXPERT_ID and clean == 0
    for g, w in zip(got, want):
        assert bool((g[-PAST:] == 7).all())
        if call == "down_combine":               # atomic sums: the order of a token's rows varies
            torch.testing.assert_close(g, w, rtol=2 ** -7, atol=1e-3)
        else:
            assert torch.equal(g, w)
