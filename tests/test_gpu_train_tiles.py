"""The training and 4-bit products over enough tiles that every CTA (or pair)
takes at least three, with ragged and empty segments (needs a B200): the hand-over of
the accumulators from tile to tile, the stages carried on across tiles, the
chunked order of a long segment's tiles, and the wide tiles of d_a on both
weight layouts. Formulas and tolerances are those of the smaller tests."""
import pytest
import torch

import mx_util as X
import test_gpu_mxfp4 as M
import test_gpu_train as T
from mixture_experts_layer_limited_b200 import native as N
from train_util import BF16_U, F32_U, F64, ffn_forward

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16

# rows of 64 experts; on average at most 16 (tiles of 32 rows), at most 32 (64) and more (192)
FEW = [16, 0, 5, 31, 32, 33, 1, 17, 0, 2, 15, 40, 3, 16, 8, 12] * 4
SOME = [64, 0, 17, 33, 1, 65, 16, 48, 31, 3, 63, 0, 20, 50, 32, 8] * 4
MANY = [192, 0, 193, 5, 400, 64, 1, 33, 97, 16, 0, 112, 3, 80, 17, 250] * 3 + [1, 1600, 0, 1537, 2, 1536] + [9, 0] * 5
# the shape of the experts: tiles of gate/up and of down are those of their row blocks eight times over
LAYERS = [(FEW, 256, 1024, 2048, 128), (SOME, 256, 1024, 2048, 128), (MANY, 256, 1024, 2048, 128)]


def _tiles(counts, blocks):
    twice = 2 * -(-sum(counts) // len(counts))
    most = 32 if twice <= 32 else 64 if twice <= 64 else 192
    return sum(-(-n // most) for n in counts) * blocks


@pytest.mark.parametrize("counts,H,I", [(c, H, I) for c, H, I, _, _ in LAYERS])
def test_4bit_gate_up_of_many_tiles(counts, H, I):
    assert _tiles([3] + counts, I // 128) >= 3 * 148
    M.test_gate_up_product(counts, H, I)


@pytest.mark.parametrize("counts,H,I", [(c, H, I) for c, _, _, H, I in LAYERS])
def test_4bit_down_of_many_tiles(counts, H, I):
    assert _tiles([3] + counts, H // 256) >= 3 * 148
    M.test_down_product(counts, H, I)


@pytest.mark.parametrize("counts", [FEW, SOME, MANY])
def test_4bit_block_of_many_tiles_twice(counts):
    """Two runs agree bit for bit."""
    H, I = 2048, 1024
    c, off, R, E = M._layer(counts, H, 128, seed=5)
    g = M._gen(7)
    code = lambda *s: torch.randint(0, 256, s, generator=g, device=DEV, dtype=torch.uint8)
    scale = lambda *s: torch.randint(118, 124, s, generator=g, device=DEV, dtype=torch.uint8)
    w = dict(w13=code(E, 2 * I, H // 2), w2=code(E, H, I // 2))
    s = dict(w13_scale=scale(E, 2 * I // 128, H // 128, 512), w2_scale=scale(E, H // 128, I // 128, 512),
             a_scale=X.row_scale_words(c["xs"]))
    a, offs = X.pack(c["x"]), torch.tensor(off, dtype=torch.int32, device=DEV)
    runs = []
    for _ in range(2):
        h = torch.empty(R, I // 2, dtype=torch.uint8, device=DEV)
        hs = torch.empty(I // 128, R, 4, dtype=torch.uint8, device=DEV)
        out = torch.empty(R, H, dtype=BF, device=DEV)
        N.moe_grouped_swiglu(R, H, w["w13"], w["w2"], N.MOE_MXFP4, E, I, a, offs, c["row_w"], h, out, h_scale_ws=hs, **s)
        runs.append((h, hs, out))
    for x, y in zip(*runs):
        assert torch.equal(x, y)


# lengths on both sides of the 32-row step, of the 256-row tile and of eight row blocks (2048 rows)
LENGTHS = [33, 0, 256, 257, 1, 300, 32, 0, 129, 17, 513, 64, 0, 200, 31, 96, 255, 2, 40, 128] * 2


@pytest.mark.parametrize("tiled", [False, True])
@pytest.mark.parametrize("counts,H,I", [(LENGTHS, 256, 1920), ([2048, 0, 2049, 5, 2500], 256, 2048)])
def test_forward_of_many_tiles(counts, H, I, tiled):
    assert sum(-(-n // 256) for n in counts) * -(-I // 256) >= 3 * 74
    c, off, R, E = T._case(counts, H, I, seed=61, lead=2, behind=3)
    w13 = T._tiled(c, E, I, H)[0] if tiled else c["w13"]
    offs = torch.tensor(off, dtype=torch.int32, device=DEV)
    runs = []
    for _ in range(2):
        h = torch.full((R, I), 7.0, dtype=BF, device=DEV)
        gu = torch.full((R, 2 * I), 7.0, dtype=BF, device=DEV)
        N.moe_gate_up_swiglu_train(R, H, w13, E, I, c["a"], offs, h, gu, tiled=tiled)
        runs.append((h, gu))
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])
    plain = torch.full((R, I), 7.0, dtype=BF, device=DEV)
    N.moe_gate_up_swiglu(R, H, w13, N.MOE_BF16, E, I, c["a"], offs, plain, tiled=tiled)
    assert torch.equal(h, plain)                     # the inference forward's h, bit for bit
    lo, hi = off[0], off[-1]
    assert bool((gu[:lo] == 7).all()) and bool((gu[hi:] == 7).all())
    ref = ffn_forward(c["a"], c["w13"], c["w2"], off, c["row_w"])[0][lo:hi]
    mag = torch.cat([c["a"][off[e]:off[e + 1]].to(F64).abs() @ c["w13"][e].to(F64).abs().T for e in range(E)])
    err = (gu[lo:hi].to(F64) - ref).abs()
    assert bool((err <= BF16_U * ref.abs() * 1.01 + H * F32_U * mag).all())


@pytest.mark.parametrize("tiled", [False, True])
@pytest.mark.parametrize("counts,H,I", [(LENGTHS, 2816, 640), ([9, 0, 2600, 1, 2049], 2816, 384)])
def test_backward_of_many_wide_tiles(counts, H, I, tiled):
    """d_a in tiles of 512 features, the last one half empty (H an odd multiple of
    256), on both weight layouts; dh0 in parts."""
    wide = sum(-(-n // 256) for n in counts) * -(-H // 512)
    assert 2 * I > 512 and H % 512 == 256 and wide >= (3 * 74 if len(counts) > 9 else 74)
    c, off, R, E = T._case(counts, H, I, seed=67)
    o = T._backward(c, off, R, E, H, I, tiled=tiled)
    T._check(o, c, off, H, I)
    again = T._backward(c, off, R, E, H, I, tiled=tiled)
    for k, v in o.items():
        assert torch.equal(v, again[k])
