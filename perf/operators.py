"""The training and 4-bit operators of the MoE layer, as a user's program runs them: the calls of libmoe's Python binding
(`own` true) beside a plain form in elementary torch operations.

  forward   the gated feed-forward block of the experts for training: h = SiLU(a w1^T) * (a w3^T) per expert segment, and the
            pre-activations that its backward pass needs
  backward  that block's and the down projection's backward pass: gradients of the rows, of both weight matrices and of the
            routing weights
  router    the backward pass of the routing weights and of the gate projection
  mxfp4     rows quantised to microscaled 4-bit floating point (E2M1 values, one power-of-two scale per 32) and read back
  ffn4      the experts' feed-forward block with 4-bit weights and activations, its input quantised on the way
"""
import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
DEV = "cuda"


def listed():
    return [
        # the tiny layer of the tests: a call of a few microseconds, where launches count
        dict(name="forward tiny", kind="forward", T=64, k=4, E=16, H=256, I=128, skew=0.0),
        # a V3 layer's share of 32 experts at V3's 256 rows per expert: an ordinary training step
        dict(name="forward v3 e32", kind="forward", T=1024, k=8, E=32, H=7168, I=2048, skew=0.3),
        dict(name="backward tiny", kind="backward", T=64, k=4, E=16, H=256, I=128, skew=0.0),
        # V2-Lite's whole layer on a micro-batch of odd length, loads uneven: ragged segments
        dict(name="backward v2lite odd", kind="backward", T=999, k=6, E=64, H=2048, I=1408, skew=0.8),
        # V2-Lite's layer at its full batch
        dict(name="backward v2lite", kind="backward", T=4096, k=6, E=64, H=2048, I=1408, skew=0.3),
        dict(name="backward v3 e32", kind="backward", T=1024, k=8, E=32, H=7168, I=2048, skew=0.3),
        # V2-Lite's router on an odd batch (softmax), V3's on a full one (sigmoid, renormalised)
        dict(name="router v2lite odd", kind="router", T=1001, k=6, E=64, H=2048, scoring="softmax", norm=False, scale=1.0),
        dict(name="router v3", kind="router", T=8192, k=8, E=256, H=7168, scoring="sigmoid", norm=True, scale=2.5),
        # a decode batch's rows gathered by expert while they are quantised; a prefill batch's rows
        dict(name="mxfp4 rows gathered", kind="mxfp4", T=33, k=6, H=2048, gather=True),
        dict(name="mxfp4 rows", kind="mxfp4", T=4096, k=1, H=7168, gather=False),
        # V3's decode (8 rows per expert) on 64 of its experts: the weights' bytes bound it
        dict(name="ffn4 v3 decode", kind="ffn4", T=64, k=8, E=64, H=7168, I=2048, skew=0.0),
        # V3's prefill share: 256 rows per expert
        dict(name="ffn4 v3 e32", kind="ffn4", T=1024, k=8, E=32, H=7168, I=2048, skew=0.3),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["forward", "backward", "backward", "router", "mxfp4", "ffn4", "ffn4"])
    H = 256 * _spread(rng, 1, 28)
    if kind == "router":
        E = 16 * rng.choice([1, 2, 4, 8, 10, 16])
        soft = rng.random() < 0.5
        k = rng.randint(1, 8)  # renormalising a single weight leaves nothing to train
        return dict(kind=kind, T=_spread(rng, 1, 8192), k=k, E=E, H=H, scoring="softmax" if soft else "sigmoid",
                    norm=k > 1 and rng.random() < 0.5, scale=rng.choice([1.0, 2.5]))
    if kind == "mxfp4":
        gather = rng.random() < 0.5
        k = rng.choice([1, 4, 6, 8]) if gather else 1
        return dict(kind=kind, T=max(1, min(_spread(rng, 1, 4096), 4096 * 7168 // (k * H))), k=k, H=H, gather=gather)
    I = 128 * _spread(rng, 1, 16)
    E = min(rng.choice([4, 8, 16, 32, 64]), 32 * 7168 * 2048 // (H * I))
    k = rng.choice([1, 2, 4, 6, 8])
    k = min(k, E)
    most = min(32768, 8192 * 7168 * 2048 // (H * I)) // k
    return dict(kind=kind, T=_spread(rng, 1, max(1, most)), k=k, E=E, H=H, I=I, skew=rng.choice([0.0, 0.3, 0.8]))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape, std=1.0, dtype=BF16):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def _weights(g, *shape):
    w = torch.empty(*shape, dtype=BF16, device=DEV)
    for e in range(shape[0]):
        w[e] = _normal(g, *shape[1:], std=0.02)
    return w


def _routes(g, T, k, E, skew):
    """Expert ids by top-k of random logits (uneven loads with `skew`), and the expert-ordered rows they give."""
    logits = torch.randn(T, E, generator=g, device=DEV) + skew * torch.randn(E, generator=g, device=DEV)
    score, ids = logits.topk(k, dim=1)
    flat = ids.reshape(-1)
    order = flat.argsort(stable=True)
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = counts.cumsum(0)
    weight = score.softmax(1).reshape(-1)[order].contiguous()
    return dict(offsets=offsets, src_token=(order // k).to(torch.int32), row_w=weight, cap=int(counts.max()))


def _blocks_of_scales(s):
    """Scales [E, N, K/32] in the order in which the kernels read a weight matrix's: per 128 rows and 128 columns, row r's
    four bytes at (r % 32) * 16 + (r / 32) * 4."""
    E, N, S = s.shape
    return s.view(E, N // 128, 4, 32, S // 4, 4).permute(0, 1, 4, 3, 2, 5).contiguous()


def _plain_of_blocks(b):
    """The scales [E, N, K/32] of _blocks_of_scales."""
    E, n, s = b.shape[:3]
    return b.permute(0, 1, 4, 3, 2, 5).reshape(E, n * 128, s * 4)


def _weights4(g, E, N, K):
    """4-bit weights as a program holds them after loading: packed codes [E, N, K/2] and their scales."""
    q = torch.empty(E, N, K // 2, dtype=torch.uint8, device=DEV)
    s = torch.empty(E, N, K // 32, dtype=torch.uint8, device=DEV)
    for e in range(E):
        code, scale = _mx_codes(_normal(g, N, K, std=0.02).float())
        q[e] = code[:, 0::2] | (code[:, 1::2] << 4)
        s[e] = scale
    return q, _blocks_of_scales(s)


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    kind, T, k, H = c["kind"], c["T"], c["k"], c["H"]
    R = T * k
    s = dict(c=c, kind=kind, R=R)
    if kind == "mxfp4":
        s["x"] = _normal(g, T, H) * torch.exp2(torch.randint(-6, 7, (T, 1), generator=g, device=DEV).to(BF16))
        s["src_token"] = (torch.randperm(R, generator=g, device=DEV) % T).to(torch.int32) if c["gather"] else None
        s["q"] = torch.empty(R, H // 2, dtype=torch.uint8, device=DEV)
        s["scale"] = torch.empty(H // 128, R, 4, dtype=torch.uint8, device=DEV)
        s["value"] = torch.empty(R, H, dtype=BF16, device=DEV)
        return s
    E = c["E"]
    if kind == "router":
        s["logits"] = _normal(g, T, E, std=0.02 * math.sqrt(H), dtype=F32)
        s["ids"] = s["logits"].topk(k, dim=1)[1].to(torch.int32)
        order = s["ids"].reshape(-1).argsort(stable=True)
        s["slot_to_row"] = torch.empty(R, dtype=torch.int32, device=DEV)
        s["slot_to_row"][order] = torch.arange(R, dtype=torch.int32, device=DEV)
        s["d_row_w"] = _normal(g, R, std=0.1, dtype=F32)
        s["x"], s["gate"] = _normal(g, T, H), _normal(g, E, H, std=0.02)
        s["dx_in"] = _normal(g, T, H, std=1e-3)
        s["d_logits"] = torch.empty(T, E, dtype=F32, device=DEV)
        s["d_logits16"] = torch.empty(T, E, dtype=BF16, device=DEV)
        s["dx"], s["d_gate"] = torch.empty_like(s["dx_in"]), torch.empty_like(s["gate"])
        return s
    I = c["I"]
    s.update(_routes(g, T, k, E, c["skew"]))
    if kind == "ffn4":
        s["x"] = _normal(g, T, H)
        s["w13"], s["w13_scale"] = _weights4(g, E, 2 * I, H)
        s["w2"], s["w2_scale"] = _weights4(g, E, H, I)
        s["q"] = torch.empty(R, H // 2, dtype=torch.uint8, device=DEV)
        s["scale"] = torch.empty(H // 128, R, 4, dtype=torch.uint8, device=DEV)
        s["h"] = torch.empty(R, I // 2, dtype=torch.uint8, device=DEV)
        s["h_scale"] = torch.empty(I // 128, R, 4, dtype=torch.uint8, device=DEV)
        s["out"] = torch.empty(R, H, dtype=BF16, device=DEV)
        return s
    s["a"], s["w13"] = _normal(g, R, H), _weights(g, E, 2 * I, H)
    if kind == "forward":
        s["h"] = torch.empty(R, I, dtype=BF16, device=DEV)
        s["gu"] = torch.empty(R, 2 * I, dtype=BF16, device=DEV)
        return s
    # backward: the pre-activations saved by the forward, and the gradient of the rows' outputs
    s["w2"] = _weights(g, E, H, I)
    s["gu"] = _normal(g, R, 2 * I, std=0.02 * math.sqrt(H))
    s["d_out"] = _normal(g, R, H, std=1e-3)
    s["d_a"], s["d_w13"], s["d_w2"] = (torch.empty_like(s[n]) for n in ("a", "w13", "w2"))
    s["d_row_w"] = torch.empty(R, dtype=F32, device=DEV)
    # what a program keeps for the call: sized by the rows alone (the intermediates' gradients and their partial sums)
    s["workspace"] = torch.empty(R * (6 * I + I // 8) + 1024, dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    return (_own if own else _plain)(state)


def _own(s):
    from mixture_experts_layer_limited_b200 import native as N
    c, R, H = s["c"], s["R"], s["c"]["H"]
    if s["kind"] == "forward":
        N.moe_gate_up_swiglu_train(R, H, s["w13"], c["E"], c["I"], s["a"], s["offsets"], s["h"], s["gu"])
        return dict(h=s["h"], gu=s["gu"])
    if s["kind"] == "backward":
        N.moe_swiglu_ffn_backward(R, H, s["w13"], s["w2"], c["E"], c["I"], s["a"], s["gu"], s["d_out"], s["offsets"], s["row_w"],
                                  s["d_a"], s["d_w13"], s["d_w2"], s["d_row_w"], s["workspace"])
        return dict(d_a=s["d_a"], d_w13=s["d_w13"], d_w2=s["d_w2"], d_row_w=s["d_row_w"])
    if s["kind"] == "router":
        N.moe_route_backward(c["T"], c["E"], c["k"], N.MOE_SOFTMAX if c["scoring"] == "softmax" else N.MOE_SIGMOID, c["norm"],
                             c["scale"], s["logits"], s["ids"], s["d_row_w"], s["slot_to_row"], s["d_logits"], s["d_logits16"])
        N.moe_gate_backward(c["T"], H, c["E"], s["d_logits16"], s["x"], s["gate"], s["dx_in"], s["dx"], s["d_gate"])
        return dict(d_logits=s["d_logits"], dx=s["dx"], d_gate=s["d_gate"])
    if s["kind"] == "mxfp4":
        N.moe_quantize_mxfp4_rows(R, H, s["x"], c["T"], s["src_token"], s["q"], s["scale"])
        N.moe_dequantize_mxfp4_rows(R, H, s["q"], s["scale"], s["value"])
        return s["value"]
    N.moe_quantize_mxfp4_rows(R, H, s["x"], c["T"], s["src_token"], s["q"], s["scale"])
    N.moe_grouped_swiglu(R, H, s["w13"], s["w2"], N.MOE_MXFP4, c["E"], c["I"], s["q"], s["offsets"], s["row_w"], s["h"], s["out"],
                         w13_scale=s["w13_scale"], w2_scale=s["w2_scale"], a_scale=s["scale"], h_scale_ws=s["h_scale"])
    return s["out"]


def _seats(s):
    """(expert, place in its segment) of every row."""
    row = torch.arange(s["R"], device=DEV)
    e = torch.searchsorted(s["offsets"][1:].long(), row, right=True)
    return e, row - s["offsets"].long()[e]


def _pad(s, seats, rows):
    """Rows [R, n] as [E, most rows of an expert, n] in fp32, zeros behind each segment."""
    p = torch.zeros(s["c"]["E"], s["cap"], rows.shape[1], device=DEV)
    p[seats] = rows.float()
    return p


def _pow2(e):
    """2^e in fp32, exactly, for whole e of [-127, 127] (a power function rounds)."""
    return ((e.long() + 1023) << 52).view(F64).float()


def _mx_codes(v):
    """fp32 rows -> E2M1 codes (a byte each) and E8M0 scale bytes per 32: the scale is 2^(floor(log2 amax) - 2), an all-zero
    block's 1; a code is the nearest value of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to the even code, above 6 to 6)."""
    b = v.view(v.shape[0], -1, 32)
    amax = b.abs().amax(-1)
    e = (torch.frexp(amax)[1] - 3).clamp(-127, 125)
    e = torch.where(amax == 0, torch.zeros_like(e), e)
    a = b.abs() * _pow2(-e).unsqueeze(-1)
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)).to(torch.uint8)
    code = code | (torch.signbit(b).to(torch.uint8) << 3)
    return code.view(v.shape), (e + 127).to(torch.uint8)


def _mx_values(code, scale):
    """The fp32 values of E2M1 codes [.., K] (a byte each) with E8M0 scale bytes [.., K/32]."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=DEV)
    v = grid[code.int()].view(*scale.shape, 32)
    return (v * _pow2(scale.int() - 127).unsqueeze(-1)).view(code.shape)


def _mx_weights(q, blocks):
    return _mx_values(torch.stack([q & 15, q >> 4], -1).view(*q.shape[:-1], -1), _plain_of_blocks(blocks))


def _plain(s):
    c, R = s["c"], s["R"]
    if s["kind"] == "mxfp4":
        x = s["x"].float() if s["src_token"] is None else s["x"].float()[s["src_token"].long()]
        code, scale = _mx_codes(x)
        return _mx_values(code, scale).to(BF16)
    if s["kind"] == "router":
        d_w = s["d_row_w"][s["slot_to_row"].long()].view(c["T"], c["k"])
        ids, l = s["ids"].long(), s["logits"]
        if c["scoring"] == "softmax":
            e = torch.exp(l - l.amax(1, keepdim=True))
            p = e / e.sum(1, keepdim=True)
        else:
            p = 1 / (1 + torch.exp(-l))
        w = p.gather(1, ids)
        if c["norm"]:
            total = w.sum(1, keepdim=True)
            d_s = c["scale"] / total * (d_w - (d_w * w).sum(1, keepdim=True) / total)
        else:
            d_s = c["scale"] * d_w
        d = torch.zeros_like(l).scatter(1, ids, d_s)
        d = p * (d - (d_s * w).sum(1, keepdim=True)) if c["scoring"] == "softmax" else p * (1 - p) * d
        return dict(d_logits=d, dx=(s["dx_in"].float() + d @ s["gate"].float()).to(BF16), d_gate=(d.T @ s["x"].float()).to(BF16))
    seats, I = _seats(s), c["I"]
    if s["kind"] == "forward":
        gu = torch.bmm(_pad(s, seats, s["a"]), s["w13"].float().transpose(1, 2))[seats]
        g, u = gu[:, :I], gu[:, I:]
        return dict(h=(g / (1 + torch.exp(-g)) * u).to(BF16), gu=gu.to(BF16))
    if s["kind"] == "backward":
        g, u = s["gu"][:, :I].float(), s["gu"][:, I:].float()
        d_out, w = _pad(s, seats, s["d_out"]), s["row_w"].unsqueeze(1)
        sig = 1 / (1 + torch.exp(-g))
        h = g * sig * u
        d_h = torch.bmm(d_out, s["w2"].float())[seats]
        d_row_w = (d_h * h).sum(1)
        d_h = d_h * w
        d_gu = _pad(s, seats, torch.cat([d_h * u * sig * (1 + g * (1 - sig)), d_h * g * sig], 1))
        return dict(d_a=torch.bmm(d_gu, s["w13"].float())[seats].to(BF16),
                    d_w13=torch.bmm(d_gu.transpose(1, 2), _pad(s, seats, s["a"])).to(BF16),
                    d_w2=torch.bmm(d_out.transpose(1, 2), _pad(s, seats, h * w)).to(BF16), d_row_w=d_row_w)
    code, scale = _mx_codes(s["x"].float())
    a = _pad(s, seats, _mx_values(code, scale)[s["src_token"].long()])
    gu = torch.bmm(a, _mx_weights(s["w13"], s["w13_scale"]).transpose(1, 2))[seats]
    g, u = gu[:, :I], gu[:, I:]
    h = _pad(s, seats, _mx_values(*_mx_codes(g / (1 + torch.exp(-g)) * u)))
    out = torch.bmm(h, _mx_weights(s["w2"], s["w2_scale"]).transpose(1, 2))[seats]
    return (out * s["row_w"].unsqueeze(1)).to(BF16)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    T, k, H = c["T"], c["k"], c["H"]
    R = T * k
    if c["kind"] == "mxfp4":
        return {"bytes": 2 * T * H + 2 * R * H + R * H // 32, "flops": 0}
    E = c["E"]
    if c["kind"] == "router":
        read = 4 * T * (E if c["scoring"] == "softmax" else k) + 12 * R + 4 * T * H + 2 * E * H
        return {"bytes": read + 4 * T * E + 2 * T * H + 2 * E * H, "flops": 4 * T * E * H}
    I, used = c["I"], min(E, R)
    if c["kind"] == "forward":
        return {"bytes": 2 * used * 2 * I * H + 2 * R * (H + 3 * I), "flops": 4 * R * H * I}
    if c["kind"] == "backward":
        return {"bytes": 2 * 3 * used * I * H + 2 * 3 * E * I * H + 2 * R * (3 * H + 2 * I) + 8 * R, "flops": 12 * R * H * I}
    return {"bytes": 3 * used * I * H * 17 // 32 + 2 * T * H + 2 * R * H + 8 * R, "flops": 6 * R * H * I}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c, R = s["c"], s["R"]
    if s["kind"] == "mxfp4":
        rows = s["x"] if s["src_token"] is None else s["x"].index_select(0, s["src_token"].long())
        return _mx64(rows.double())
    if s["kind"] == "router":
        T, k = c["T"], c["k"]
        z = s["logits"].double().requires_grad_()
        score = torch.softmax(z, 1) if c["scoring"] == "softmax" else torch.sigmoid(z)
        w = torch.take_along_dim(score, s["ids"].long(), 1)
        w = (w / w.sum(1, keepdim=True) if c["norm"] else w) * c["scale"]
        up = torch.stack([s["d_row_w"].double()[s["slot_to_row"].long()[j::k]] for j in range(k)], 1)
        d, = torch.autograd.grad((w * up).sum(), z)
        return dict(d_logits=d, dx=s["dx_in"].double().addmm(d, s["gate"].double()), d_gate=d.t().mm(s["x"].double()))
    H, I, E = c["H"], c["I"], c["E"]
    ends = s["offsets"].tolist()
    new = lambda *n: torch.zeros(*n, dtype=F64, device=DEV)  # noqa: E731
    if s["kind"] == "forward":
        h, gu = new(R, I), new(R, 2 * I)
        for e in range(E):
            at = slice(ends[e], ends[e + 1])
            gu[at] = s["a"][at].double() @ s["w13"][e].double().T
            h[at] = torch.nn.functional.silu(gu[at, :I]) * gu[at, I:]
        return dict(h=h, gu=gu)
    if s["kind"] == "backward":
        d_a, d_row_w, d_w13, d_w2 = new(R, H), new(R), s["w13"].new_empty(0), None
        w13_grads, w2_grads = [], []
        for e in range(E):
            at = slice(ends[e], ends[e + 1])
            z = s["gu"][at].double().requires_grad_()
            w2 = s["w2"][e].double().requires_grad_()
            w = s["row_w"][at].double().requires_grad_()
            out = w[:, None] * ((torch.nn.functional.silu(z[:, :I]) * z[:, I:]) @ w2.T)
            dz, dw2, d_row_w[at] = torch.autograd.grad(out, (z, w2, w), s["d_out"][at].double())
            d_a[at] = dz @ s["w13"][e].double()
            w13_grads.append((dz.T @ s["a"][at].double()).float())
            w2_grads.append(dw2.float())
        # kept in 32 bits, far finer than the bf16 gradients that they are held against
        d_w13, d_w2 = torch.stack(w13_grads), torch.stack(w2_grads)
        return dict(d_a=d_a, d_w13=d_w13, d_w2=d_w2, d_row_w=d_row_w)
    x, out = _mx64(s["x"].double()), new(R, H)
    for e in range(E):
        at = slice(ends[e], ends[e + 1])
        a = x.index_select(0, s["src_token"][at].long())
        gu = a @ _weight64(s["w13"][e], s["w13_scale"][e]).T
        h = _mx64(torch.nn.functional.silu(gu[:, :I]) * gu[:, I:])
        out[at] = s["row_w"][at].double()[:, None] * (h @ _weight64(s["w2"][e], s["w2_scale"][e]).T)
    return out


def _mx64(v):
    """fp64 rows -> the values that their 4-bit codes stand for: the nearest grid point by distance."""
    if v.numel() == 0:
        return v
    b = v.reshape(-1, 32)
    amax = b.abs().max(1, keepdim=True)[0]
    e = (torch.where(amax > 0, amax, torch.full_like(amax, 4.0)).view(torch.int64) >> 52) - 1023 - 2  # the exponent's bits
    e = e.clamp(-127, 125)
    unit = ((e + 1023) << 52).view(F64)  # 2^e
    a = b.abs() / unit
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    near = torch.clamp(torch.round(a / step) * step, max=6.0)  # round() takes ties to even multiples: the even codes
    return torch.copysign(near * unit, b).reshape(v.shape)


def _weight64(q, blocks):
    n, s = blocks.shape[:2]
    N, K = n * 128, s * 128
    nibble = torch.empty(N, K, dtype=torch.int64, device=DEV)
    nibble[:, 0::2], nibble[:, 1::2] = (q & 15).long(), (q >> 4).long()
    m = nibble & 7
    size = torch.where(m < 2, 0.5 * m, (1 + 0.5 * (m & 1)) * (1 << (m >> 1)) * 0.5)
    scale = torch.empty(N, K // 32, dtype=F64, device=DEV)
    for j in range(4):  # rows 32j .. 32j+31 of every block of 128
        scale.view(n, 4, 32, s, 4)[:, j] = blocks[:, :, :, j].permute(0, 2, 1, 3).double()
    unit = ((scale.long() + 1023 - 127) << 52).view(F64)
    value = torch.where(nibble > 7, -size, size).view(N, -1, 32) * unit.unsqueeze(-1)
    return value.reshape(N, K)
