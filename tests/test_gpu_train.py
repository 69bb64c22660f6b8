"""The training operators of libmoe against float64 formulas (needs a B200):
the experts' forward that saves its pre-activations, their backward pass, the
router's and the gate's. Tolerances: tests/train_util.backward_tolerance."""
import pytest
import torch

from mixture_experts_layer_limited_b200 import native as N
from train_util import (BF16_U, F32_U, F64, backward_tolerance, ffn_backward, ffn_forward, route_weights, segments)

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _case(counts, H, I, seed, lead=0, behind=0):
    """Inputs over segments of `counts` rows; `lead` / `behind` rows of NaN
    before the first and after the last segment belong to nobody."""
    g = _gen(seed)
    off = segments(counts, lead)
    R, E = off[-1] + behind, len(counts)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=g, device=DEV) * std).to(BF)
    c = dict(a=n(R, H), gu=n(R, 2 * I, std=1.5), d_out=n(R, H, std=0.1), w13=n(E, 2 * I, H, std=0.05),
             w2=n(E, H, I, std=0.05), row_w=torch.rand(R, generator=g, device=DEV) + 0.1)
    for k in ("a", "gu", "d_out", "row_w"):
        c[k][:lead] = float("nan")
        c[k][off[-1]:] = float("nan")
    return c, off, R, E


def _tiled(c, E, I, H):
    t13, t2 = torch.empty_like(c["w13"]), torch.empty_like(c["w2"])
    N.moe_tile_ffn_weights(H, c["w13"], c["w2"], E, I, t13, t2)
    return t13, t2


def _backward(c, off, R, E, H, I, tiled=False, f32=False, accumulate=False, init=None, row_w=True, want=None):
    gt = torch.float32 if f32 else BF
    o = dict(d_a=torch.full((R, H), 7.0, dtype=BF, device=DEV), d_w13=torch.full((E, 2 * I, H), 7.0, dtype=gt, device=DEV),
             d_w2=torch.full((E, H, I), 7.0, dtype=gt, device=DEV), d_row_w=torch.full((R,), 7.0, device=DEV))
    if init is not None:
        o["d_w13"].copy_(init[0])
        o["d_w2"].copy_(init[1])
    if want is not None:
        o = {k: v if k in want else None for k, v in o.items()}
    w13, w2 = _tiled(c, E, I, H) if tiled else (c["w13"], c["w2"])
    ws = torch.empty(N.moe_swiglu_ffn_backward_workspace_size(R, I), dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    offs = torch.tensor(off, dtype=torch.int32, device=DEV) if off is not None else None
    N.moe_swiglu_ffn_backward(R, H, w13, w2, E, I, c["a"], c["gu"], c["d_out"], offs, c["row_w"] if row_w else None,
                              o["d_a"], o["d_w13"], o["d_w2"], o["d_row_w"], ws,
                              grad_dtype=N.MOE_F32 if f32 else N.MOE_BF16, accumulate=accumulate, dev_status=status,
                              tiled=tiled)
    assert N.moe_read_device_status(status) == 0
    return o


def _check(o, c, off, H, I, f32=False):
    row_w = c["row_w"]
    ref, mag, fp = ffn_backward(c["a"], c["gu"], c["d_out"], c["w13"], c["w2"], off, row_w)
    lo, hi = off[0], off[-1]
    for name, got in o.items():
        if got is None:
            continue
        dt = got.dtype
        rows = max(off[i + 1] - off[i] for i in range(len(off) - 1))
        tol = backward_tolerance(name, ref[name], mag[name], fp.get(name), H, I, rows, dt)
        err = (got.to(F64) - ref[name]).abs()
        if name in ("d_a", "d_row_w"):
            assert bool((got[:lo] == 7).all()) and bool((got[hi:] == 7).all()), f"{name}: rows of nobody were written"
            err, tol = err[lo:hi], tol[lo:hi]
        assert bool((err <= tol + 1e-30).all()), (name, float((err - tol).max()), float(err.max()))


SHAPES = [
    # counts, H, I: lengths around the 16-row MMA step, the 64-row K block and the 256-row tile, empty experts
    ([5, 0, 16, 1], 256, 128),
    ([64, 65, 0, 17, 63], 512, 384),
    ([256, 0, 257, 15], 256, 256),
    ([0, 0, 3], 768, 640),
    ([1], 256, 128),
    ([300, 1, 129], 1024, 1408),
]


@pytest.mark.parametrize("tiled", [False, True])
@pytest.mark.parametrize("counts,H,I", SHAPES)
def test_backward_matches_formula(counts, H, I, tiled):
    c, off, R, E = _case(counts, H, I, seed=len(counts) * 7 + H)
    _check(_backward(c, off, R, E, H, I, tiled=tiled), c, off, H, I)


def test_backward_leaves_rows_of_nobody_alone():
    """NaN rows before the first and behind the last segment: nothing of them
    enters a gradient, and their outputs stay as they were."""
    c, off, R, E = _case([5, 0, 33, 70], 256, 128, seed=3, lead=9, behind=21)
    _check(_backward(c, off, R, E, 256, 128), c, off, 256, 128)


def test_backward_without_any_row():
    """No expert has a row: the weights' gradients are zero (left alone when
    accumulating), nothing else is written."""
    H, I = 256, 128
    c, off, R, E = _case([0, 0, 0], H, I, seed=14, lead=1, behind=2)
    o = _backward(c, off, R, E, H, I)
    assert bool((o["d_w13"] == 0).all()) and bool((o["d_w2"] == 0).all())
    assert bool((o["d_a"] == 7).all()) and bool((o["d_row_w"] == 7).all())
    init = (torch.full((E, 2 * I, H), 3.0, device=DEV), torch.full((E, H, I), 4.0, device=DEV))
    o = _backward(c, off, R, E, H, I, f32=True, accumulate=True, init=init)
    assert bool((o["d_w13"] == 3).all()) and bool((o["d_w2"] == 4).all())


def test_segments_outside_the_rows_are_cut_and_flagged():
    """offsets past the rows there are: nothing is read or written outside."""
    H, I = 256, 128
    c, off, R, E = _case([20, 30], H, I, seed=15)
    good = _backward(c, off, R, E, H, I)
    offs = torch.tensor([0, 20, 10_000], dtype=torch.int32, device=DEV)
    o = {k: torch.zeros_like(v) for k, v in good.items()}
    ws = torch.empty(N.moe_swiglu_ffn_backward_workspace_size(R, I), dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    N.moe_swiglu_ffn_backward(R, H, c["w13"], c["w2"], E, I, c["a"], c["gu"], c["d_out"], offs, c["row_w"], o["d_a"],
                              o["d_w13"], o["d_w2"], o["d_row_w"], ws, dev_status=status)
    assert N.moe_read_device_status(status) & N.MOE_DEVSTAT_BAD_EXPERT_ID
    for k in good:
        assert torch.equal(o[k], good[k])


def test_segment_that_ends_before_it_starts_is_empty_and_flagged():
    """Falling offsets: that expert has no rows (no wait runs out), the others
    keep theirs."""
    H, I = 256, 128
    c, off, R, E = _case([20, 30, 6], H, I, seed=18)
    offs = [0, 20, 5, 5]
    o = {k: torch.zeros_like(v) for k, v in _backward(c, off, R, E, H, I).items()}
    ws = torch.empty(N.moe_swiglu_ffn_backward_workspace_size(R, I), dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    N.moe_swiglu_ffn_backward(R, H, c["w13"], c["w2"], E, I, c["a"], c["gu"], c["d_out"],
                              torch.tensor(offs, dtype=torch.int32, device=DEV), c["row_w"], o["d_a"], o["d_w13"],
                              o["d_w2"], o["d_row_w"], ws, dev_status=status)
    assert N.moe_read_device_status(status) == N.MOE_DEVSTAT_BAD_EXPERT_ID
    good = _backward(c, off, R, E, H, I)
    assert torch.equal(o["d_a"][:20], good["d_a"][:20]) and torch.equal(o["d_row_w"][:5], good["d_row_w"][:5])
    for k in ("d_w13", "d_w2"):
        assert torch.equal(o[k][0], good[k][0]) and not bool(o[k][1:].any())


def test_calls_on_two_streams_at_once():
    """Two backward passes in flight at once, a workspace each, give what they
    give one after the other."""
    H, I = 512, 384
    cases = [_case([90, 7, 0, 200], H, I, seed=s) for s in (16, 17)]
    want = [_backward(c, off, R, E, H, I) for c, off, R, E in cases]
    got, streams = [], [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for s, (c, off, R, E) in zip(streams, cases):
            with torch.cuda.stream(s):
                o = {k: torch.zeros_like(v) for k, v in want[0].items()}
                ws = torch.empty(N.moe_swiglu_ffn_backward_workspace_size(R, I), dtype=torch.uint8, device=DEV)
                offs = torch.tensor(off, dtype=torch.int32, device=DEV)
                N.moe_swiglu_ffn_backward(R, H, c["w13"], c["w2"], E, I, c["a"], c["gu"], c["d_out"], offs, c["row_w"],
                                          o["d_a"], o["d_w13"], o["d_w2"], o["d_row_w"], ws)
                got.append((o, ws, offs))
        torch.cuda.synchronize()
    for (o, _, _), w in zip(got, want):
        for k in w:
            assert torch.equal(o[k], w[k])


def test_backward_nan_in_one_expert_stays_there():
    """The rows behind a segment's end are the next expert's: NaN and infinity
    in them must not reach this expert's weight gradients."""
    c, off, R, E = _case([17, 20, 31], 256, 128, seed=4)
    s = slice(off[1], off[2])
    c["a"][s] = float("nan")
    c["d_out"][s] = float("inf")
    o = _backward(c, off, R, E, 256, 128)
    for k in ("d_w13", "d_w2"):
        assert bool(torch.isfinite(o[k][0]).all()) and bool(torch.isfinite(o[k][2]).all())
        assert not bool(torch.isfinite(o[k][1]).all())
    clean, _, _, _ = _case([17, 20, 31], 256, 128, seed=4)
    p = _backward(clean, off, R, E, 256, 128)
    for e in (0, 2):
        assert torch.equal(o["d_w13"][e], p["d_w13"][e]) and torch.equal(o["d_w2"][e], p["d_w2"][e])


@pytest.mark.parametrize("accumulate", [False, True])
def test_backward_fp32_weight_gradients(accumulate):
    counts, H, I = [40, 0, 130], 512, 384
    c, off, R, E = _case(counts, H, I, seed=5)
    g = _gen(6)
    init = (torch.randn(E, 2 * I, H, generator=g, device=DEV), torch.randn(E, H, I, generator=g, device=DEV))
    o = _backward(c, off, R, E, H, I, f32=True, accumulate=accumulate, init=init)
    if accumulate:
        assert torch.equal(o["d_w13"][1], init[0][1]) and torch.equal(o["d_w2"][1], init[1][1])
        for k, i in (("d_w13", init[0]), ("d_w2", init[1])):
            # one more fp32 rounding, of a sum of at most |init| + |gradient|
            ref, mag, fp = ffn_backward(c["a"], c["gu"], c["d_out"], c["w13"], c["w2"], off, c["row_w"])
            tol = backward_tolerance(k, ref[k], mag[k], fp.get(k), H, I, max(counts), torch.float32)
            tol = tol + F32_U * (i.to(F64) + ref[k]).abs() * 2
            assert bool(((o[k].to(F64) - i.to(F64) - ref[k]).abs() <= tol).all())
        return
    _check(o, c, off, H, I)
    assert bool((o["d_w13"][1] == 0).all()) and bool((o["d_w2"][1] == 0).all())


def test_backward_long_segments_and_one_group():
    """Segments past 512 rows on average take the wide weight-gradient tile;
    offsets NULL: one group of all rows, no routing weight (the shared expert)."""
    H, I = 512, 384
    c, off, R, E = _case([900, 333], H, I, seed=8)
    _check(_backward(c, off, R, E, H, I), c, off, H, I)
    c, off, R, E = _case([1025], H, I, seed=9)
    c["row_w"].fill_(1.0)
    o = _backward(c, None, R, E, H, I, row_w=False)
    _check(o, c, off, H, I)


@pytest.mark.parametrize("f32", [False, True])
def test_backward_many_experts_of_all_lengths(f32):
    """Enough experts that a pair of SMs takes runs of weight-gradient tiles,
    with segments that fit (at most 384 rows), that do not, that end anywhere in
    a K step, and that are empty, next to one another."""
    counts = [0, 1, 15, 16, 17, 63, 64, 65, 128, 384, 385, 0, 200, 383, 400, 31, 320, 321, 48, 449, 2, 0, 96, 333]
    H, I = 1024, 1408
    c, off, R, E = _case(counts, H, I, seed=21)
    o = _backward(c, off, R, E, H, I, f32=f32)
    _check(o, c, off, H, I)
    again = _backward(c, off, R, E, H, I, f32=f32)
    for k, v in o.items():
        assert torch.equal(v, again[k])


def test_backward_outputs_on_their_own_and_twice():
    """Each output alone is what it is among all; two calls agree bit for bit."""
    H, I = 256, 384
    c, off, R, E = _case([70, 0, 19], H, I, seed=10)
    full = _backward(c, off, R, E, H, I)
    again = _backward(c, off, R, E, H, I)
    for k, v in full.items():
        assert torch.equal(v, again[k])
        assert torch.equal(_backward(c, off, R, E, H, I, want=(k,))[k], v)


@pytest.mark.parametrize("tiled", [False, True])
def test_forward_saves_preactivations(tiled):
    counts, H, I = [5, 0, 257, 40], 512, 384
    c, off, R, E = _case(counts, H, I, seed=11, lead=2, behind=3)
    w13 = _tiled(c, E, I, H)[0] if tiled else c["w13"]
    h = torch.full((R, I), 7.0, dtype=BF, device=DEV)
    gu = torch.full((R, 2 * I), 7.0, dtype=BF, device=DEV)
    offs = torch.tensor(off, dtype=torch.int32, device=DEV)
    N.moe_gate_up_swiglu_train(R, H, w13, E, I, c["a"], offs, h, gu, tiled=tiled)
    plain = torch.full((R, I), 7.0, dtype=BF, device=DEV)
    N.moe_gate_up_swiglu(R, H, w13, N.MOE_BF16, E, I, c["a"], offs, plain, tiled=tiled)
    assert torch.equal(h, plain)                     # the inference forward's h, bit for bit
    lo, hi = off[0], off[-1]
    assert bool((gu[:lo] == 7).all()) and bool((gu[hi:] == 7).all())
    ref = ffn_forward(c["a"], c["w13"], c["w2"], off, c["row_w"])[0][lo:hi]
    mag = torch.cat([c["a"][off[e]:off[e + 1]].to(F64).abs() @ c["w13"][e].to(F64).abs().T for e in range(E)])
    err = (gu[lo:hi].to(F64) - ref).abs()
    assert bool((err <= BF16_U * ref.abs() * 1.01 + H * F32_U * mag).all())


def test_forward_backward_against_differences():
    """A whole step: gradients of sum(out * v) at the saved pre-activations,
    along random directions, against central differences of the float64
    forward. The pre-activations' rounding (U_bf16 of gu, through a Lipschitz
    factor below 2 here) and the operands' bound the difference to 2 %."""
    counts, H, I = [30, 0, 21], 256, 128
    c, off, R, E = _case(counts, H, I, seed=12)
    offs = torch.tensor(off, dtype=torch.int32, device=DEV)
    h = torch.empty(R, I, dtype=BF, device=DEV)
    N.moe_gate_up_swiglu_train(R, H, c["w13"], E, I, c["a"], offs, h, c["gu"])
    o = _backward(c, off, R, E, H, I)
    g = _gen(13)
    eps = 1e-4
    names = dict(d_a="a", d_w13="w13", d_w2="w2", d_row_w="row_w")
    for gname, name in names.items():
        x = c[name].to(F64)
        # a direction with a large derivative: half along the gradient, half random
        d = torch.randn(x.shape, generator=g, device=DEV, dtype=F64)
        grad = o[gname].to(F64)
        d = d / d.norm() + grad / grad.norm()
        f = []
        for s in (1, -1):
            args = {k: v.to(F64) for k, v in c.items() if k in ("a", "w13", "w2", "row_w")}
            args[name] = x + s * eps * d
            f.append(float((ffn_forward(args["a"], args["w13"], args["w2"], off, args["row_w"])[2]
                            * c["d_out"].to(F64)).sum()))
        diff, got = (f[0] - f[1]) / (2 * eps), float((grad * d).sum())
        assert got == pytest.approx(diff, rel=2e-2), (name, got, diff)


# ------------------------------------------------------------------ router
def test_python_checks_sizes_types_and_layout():
    H, I = 256, 128
    c, off, R, E = _case([20, 30], H, I, seed=18)
    offs = torch.tensor(off, dtype=torch.int32, device=DEV)
    h, gu = torch.empty(R, I, dtype=BF, device=DEV), torch.empty(R, 2 * I, dtype=BF, device=DEV)
    call = lambda **kw: N.moe_gate_up_swiglu_train(*[{**dict(rows=R, H=H, w13=c["w13"], groups=E, I=I, a=c["a"], offsets=offs,
                                                            h=h, gu=gu), **kw}[k]
                                                     for k in ("rows", "H", "w13", "groups", "I", "a", "offsets", "h", "gu")])
    call()
    for bad in (dict(gu=gu[:-1]), dict(h=h.float()), dict(a=c["a"].cpu()), dict(offsets=offs.long()),
                dict(a=c["a"].t().contiguous().t())):
        with pytest.raises(ValueError):
            call(**bad)


ROUTES = [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)]


@pytest.mark.parametrize("scoring,norm", ROUTES)
@pytest.mark.parametrize("T,E,k", [(1, 16, 4), (33, 64, 6), (257, 256, 8), (65, 48, 16), (40, 256, 1)])
def test_route_backward(scoring, norm, T, E, k):
    g = _gen(T + E)
    logits = torch.randn(T, E, generator=g, device=DEV) * 2
    ids = torch.rand(T, E, generator=g, device=DEV).topk(k, dim=1)[1].to(torch.int32)
    dw = torch.randn(T, k, generator=g, device=DEV)
    perm = torch.randperm(T * k, generator=g, device=DEV).to(torch.int32)
    rows = torch.empty(T * k, device=DEV)
    rows[perm.long()] = dw.reshape(-1)
    x = logits.to(F64).requires_grad_()
    w = route_weights(x, ids, scoring, norm, 2.5)
    ref, = torch.autograd.grad((w * dw.to(F64)).sum(), x)
    code = N.MOE_SOFTMAX if scoring == "softmax" else N.MOE_SIGMOID
    out, out16 = torch.full((T, E), 7.0, device=DEV), torch.empty(T, E, dtype=BF, device=DEV)
    N.moe_route_backward(T, E, k, code, norm, 2.5, logits, ids, rows, perm, out, out16)
    slot = torch.empty(T, E, device=DEV)
    N.moe_route_backward(T, E, k, code, norm, 2.5, logits, ids, dw.contiguous(), None, slot)
    assert torch.equal(out, slot) and torch.equal(out16, out.to(BF))
    # every term is a product of a few factors, each good to some fp32 roundings (exp: 2 ulp; sums of E and of k
    # terms), before it cancels against the others: 64 roundings of the terms' largest magnitude
    s = torch.softmax(x, 1) if scoring == "softmax" else torch.sigmoid(x)
    sc = s.gather(1, ids.long())
    S = sc.sum(1, keepdim=True) if norm else 1.0
    most = (2.5 / S * (dw.abs().to(F64) + (dw.abs() * sc).sum(1, keepdim=True) / S)).amax(1, keepdim=True)
    assert bool(((out.to(F64) - ref).abs() <= 64 * F32_U * most * s * k + 1e-30).all())


def test_route_backward_skips_missing_experts():
    """ids of -1 (tokens without a comparable score) and ids past E count for
    nothing; the latter are flagged."""
    T, E, k = 8, 16, 4
    g = _gen(1)
    logits = torch.randn(T, E, generator=g, device=DEV)
    ids = torch.arange(k, dtype=torch.int32, device=DEV).repeat(T, 1)
    dw = torch.ones(T, k, device=DEV)
    ids[2] = -1
    out = torch.empty(T, E, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    N.moe_route_backward(T, E, k, N.MOE_SIGMOID, False, 1.0, logits, ids, dw, None, out, dev_status=status)
    assert N.moe_read_device_status(status) == 0
    assert bool((out[2] == 0).all()) and bool((out[3, :k] != 0).all())
    ids[4, 1] = E
    N.moe_route_backward(T, E, k, N.MOE_SIGMOID, False, 1.0, logits, ids, dw, None, out, dev_status=status)
    assert N.moe_read_device_status(status) & N.MOE_DEVSTAT_BAD_EXPERT_ID
    assert float(out[4, 1]) == 0 and float(out[4, 0]) != 0


@pytest.mark.parametrize("T,H,E", [(1, 256, 16), (33, 512, 64), (300, 256, 256), (1000, 1024, 48), (129, 256, 144)])
def test_gate_backward(T, H, E):
    g = _gen(T)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV).to(BF)
    dl, x, gate, dx_in = n(T, E), n(T, H), n(E, H), n(T, H)
    dx, dg = torch.empty_like(x), torch.empty_like(gate)
    N.moe_gate_backward(T, H, E, dl, x, gate, dx_in, dx, dg)
    L, X, G = dl.to(F64), x.to(F64), gate.to(F64)
    for got, ref, mag, n_terms in ((dx, dx_in.to(F64) + L @ G, dx_in.to(F64).abs() + L.abs() @ G.abs(), E + 1),
                                   (dg, L.T @ X, L.abs().T @ X.abs(), T)):
        assert bool(((got.to(F64) - ref).abs() <= BF16_U * ref.abs() * 1.01 + n_terms * F32_U * mag).all())
    # in place, without a term, and fp32 sums added to what is there
    inplace = dx_in.clone()
    N.moe_gate_backward(T, H, E, dl, x, gate, inplace, inplace, None)
    assert torch.equal(inplace, dx)
    N.moe_gate_backward(T, H, E, dl, None, gate, None, dx, None)
    assert bool(((dx.to(F64) - L @ G).abs() <= BF16_U * (L @ G).abs() * 1.01 + E * F32_U * (L.abs() @ G.abs())).all())
    acc = torch.ones(E, H, device=DEV)
    N.moe_gate_backward(T, H, E, dl, x, None, None, None, acc, grad_dtype=N.MOE_F32, accumulate=True)
    ref = L.T @ X
    assert bool(((acc.to(F64) - 1 - ref).abs() <= 2 * F32_U * (1 + ref.abs()) + T * F32_U * (L.abs().T @ X.abs())).all())


# ---------------------------- few weight-gradient tiles of many rows: split over rows
@pytest.mark.parametrize("T,H,E", [(1500, 512, 48), (1023, 256, 256), (2077, 1024, 16), (4100, 256, 176), (3001, 7168, 64)])
def test_gate_backward_of_many_rows(T, H, E):
    g = _gen(T)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV).to(BF)
    dl, x = n(T, E), n(T, H)
    ref, mag = dl.to(F64).T @ x.to(F64), dl.to(F64).abs().T @ x.to(F64).abs()
    dg = torch.empty(E, H, dtype=BF, device=DEV)
    N.moe_gate_backward(T, H, E, dl, x, None, None, None, dg)
    assert bool(((dg.to(F64) - ref).abs() <= BF16_U * ref.abs() * 1.01 + T * F32_U * mag).all())
    acc = torch.ones(E, H, device=DEV)
    for k in (1, 2):                                                      # adds again
        N.moe_gate_backward(T, H, E, dl, x, None, None, None, acc, grad_dtype=N.MOE_F32, accumulate=True)
        assert bool(((acc.to(F64) - 1 - k * ref).abs() <= 2 * k * F32_U * (1 + k * ref.abs()) + k * T * F32_U * mag).all())
    again = torch.empty_like(dg)
    N.moe_gate_backward(T, H, E, dl, x, None, None, None, again)
    assert torch.equal(dg, again)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("counts,H,I", [([1500, 601], 256, 256), ([1100], 512, 256), ([5, 2500, 0], 256, 512),
                                        ([1, 40, 1200], 256, 256)])
def test_backward_of_few_long_segments(counts, H, I, f32):
    c, off, R, E = _case(counts, H, I, seed=41)
    _check(_backward(c, off, R, E, H, I, f32=f32), c, off, H, I, f32)


@pytest.mark.parametrize("counts,H,I", [([300, 1, 17], 7168, 128), ([40, 0, 513], 5120, 384), ([9, 250], 2816, 256),
                                        ([2000, 700], 5376, 256)])
def test_backward_of_long_rows(counts, H, I):
    """dh0 summed in parts, over more tiles than there are SMs as well."""
    c, off, R, E = _case(counts, H, I, seed=47)
    _check(_backward(c, off, R, E, H, I), c, off, H, I)


@pytest.mark.parametrize("H", [768, 2048, 5120, 7168])
def test_row_weight_gradient_is_not_cut_short(H):
    """The tensor cores cut their sums towards zero. Half a unit in the last
    place, 0.72 * 2^-23 of the value on average, each 16 terms, of a sum that is
    two thirds of the last one on average: 2.9e-8 a step, 1.6e-6 for the 56
    steps of a part of 896 terms, against 1.3e-5 for 7168 in one."""
    c, off, R, E = _case([200, 56], H, 256, seed=53)
    o = _backward(c, off, R, E, H, 256)
    ref = ffn_backward(c["a"], c["gu"], c["d_out"], c["w13"], c["w2"], off, c["row_w"])[0]["d_row_w"]
    lo, hi = off[0], off[-1]
    d = o["d_row_w"].to(F64)[lo:hi] - ref[lo:hi]
    assert float(d.norm() / ref[lo:hi].norm()) < 1.6e-6


def test_split_weight_gradient_gives_up_and_recovers():
    """The wait limit in a weight gradient whose tiles several pairs share."""
    T, H, E = 2000, 512, 64
    g = _gen(43)
    dl, x = (torch.randn(T, n, generator=g, device=DEV).to(BF) for n in (E, H))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def run():
        dg = torch.zeros(E, H, dtype=BF, device=DEV)
        N.moe_gate_backward(T, H, E, dl, x, None, None, None, dg, dev_status=status)
        return dg, N.moe_read_device_status(status)
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
    assert st == 0 and torch.equal(before, after)


# -------------------------------------------------- bounded waits time out
def test_wait_limit_in_a_sum_of_parts():
    """The wait limit in a backward pass whose dh0 comes in parts."""
    H, I = 5376, 256
    c, off, R, E = _case([300, 20], H, I, seed=59)
    before = _backward(c, off, R, E, H, I)
    offs = torch.tensor(off, dtype=torch.int32, device=DEV)
    ws = torch.empty(N.moe_swiglu_ffn_backward_workspace_size(R, I), dtype=torch.uint8, device=DEV)
    status, drw = torch.zeros(1, dtype=torch.int32, device=DEV), torch.zeros(R, device=DEV)
    N.moe_set_wait_limit_ns(5)
    try:
        N.moe_swiglu_ffn_backward(R, H, c["w13"], c["w2"], E, I, c["a"], c["gu"], c["d_out"], offs, c["row_w"], None, None,
                                  None, drw, ws, dev_status=status)
        assert N.moe_read_device_status(status) == N.MOE_DEVSTAT_TIMEOUT
    finally:
        N.moe_set_wait_limit_ns(0)
    after = _backward(c, off, R, E, H, I)
    for k in before:
        assert torch.equal(before[k], after[k])


@pytest.mark.parametrize("call", ["forward", "backward", "gate"])
def test_wait_limit_runs_out_then_the_same_call_is_correct(call):
    """With a wait limit of a few nanoseconds the kernels give up at the first
    wait that does not succeed at once: they flag MOE_DEVSTAT_TIMEOUT, let
    their copies and MMAs end, free their tensor memory and return. The same
    call with the default limit then gives what it gave before."""
    H, I, counts = 512, 384, [300, 17, 0, 129]
    c, off, R, E = _case(counts, H, I, seed=31)
    offs = torch.tensor(off, dtype=torch.int32, device=DEV)
    g = _gen(32)
    dl, gate = (torch.randn(R, 48, generator=g, device=DEV)).to(BF), torch.randn(48, H, generator=g, device=DEV).to(BF)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = torch.empty(N.moe_swiglu_ffn_backward_workspace_size(R, I), dtype=torch.uint8, device=DEV)

    def run():
        if call == "forward":
            o = [torch.zeros(R, I, dtype=BF, device=DEV), torch.zeros(R, 2 * I, dtype=BF, device=DEV)]
            N.moe_gate_up_swiglu_train(R, H, c["w13"], E, I, c["a"], offs, *o, dev_status=status)
        elif call == "backward":
            o = [torch.zeros_like(c["a"]), torch.zeros_like(c["w13"]), torch.zeros_like(c["w2"]), torch.zeros(R, device=DEV)]
            N.moe_swiglu_ffn_backward(R, H, c["w13"], c["w2"], E, I, c["a"], c["gu"], c["d_out"], offs, c["row_w"], *o, ws,
                                      dev_status=status)
        else:
            o = [torch.zeros_like(c["a"]), torch.zeros_like(gate)]
            N.moe_gate_backward(R, H, 48, dl, c["a"], gate, None, *o, dev_status=status)
        return o, N.moe_read_device_status(status)
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
    for a, b in zip(before, after):
        assert torch.equal(a, b)
