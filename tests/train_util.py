"""The training operators' formulas in float64 torch (not a test module)."""
import torch

BF16_U = torch.finfo(torch.bfloat16).eps / 2    # half a step, relative
F32_U = torch.finfo(torch.float32).eps / 2
F64 = torch.float64


def segments(counts, lead=0):
    """offsets [E+1] int32 of segments of the given lengths, the first at row `lead`."""
    off = [lead]
    for n in counts:
        off.append(off[-1] + n)
    return off


def ffn_forward(a, w13, w2, offsets, row_w):
    """(gu, h, out) of the experts over their segments, float64."""
    R, I = a.shape[0], w2.shape[2]
    gu = torch.zeros(R, 2 * I, dtype=F64, device=a.device)
    h = torch.zeros(R, I, dtype=F64, device=a.device)
    out = torch.zeros(R, w2.shape[1], dtype=F64, device=a.device)
    for e in range(len(offsets) - 1):
        s = slice(offsets[e], offsets[e + 1])
        gu[s] = a[s].to(F64) @ w13[e].to(F64).T
        h[s] = gu[s, :I] * torch.sigmoid(gu[s, :I]) * gu[s, I:]
        out[s] = row_w[s].to(F64)[:, None] * (h[s] @ w2[e].to(F64).T)
    return gu, h, out


def ffn_backward(a, gu, d_out, w13, w2, offsets, row_w):
    """Gradients at the pre-activations gu, float64, and for each the sum of the
    magnitudes of its terms (what rounding errors scale with)."""
    R, H = a.shape
    E, _, I = w2.shape
    dev = a.device
    z = lambda *n: torch.zeros(*n, dtype=F64, device=dev)
    g = dict(d_a=z(R, H), d_w13=z(E, 2 * I, H), d_w2=z(E, H, I), d_row_w=z(R))
    m = {k: torch.zeros_like(v) for k, v in g.items()}
    for e in range(E):
        s = slice(offsets[e], offsets[e + 1])
        W13, W2 = w13[e].to(F64), w2[e].to(F64)
        A, D, Z, w = a[s].to(F64), d_out[s].to(F64), gu[s].to(F64), row_w[s].to(F64)[:, None]
        G, U = Z[:, :I], Z[:, I:]
        sg = torch.sigmoid(G)
        act = G * sg
        h = act * U
        dh0, dh0m = D @ W2, D.abs() @ W2.abs()
        dgf, duf = U * sg * (1 + G * (1 - sg)), act
        dgu = torch.cat([dh0 * w * dgf, dh0 * w * duf], 1)
        dgum = torch.cat([dh0m * w.abs() * (U * sg).abs() * (1 + G.abs()), dh0m * w.abs() * duf.abs()], 1)
        g["d_row_w"][s] = (h * dh0).sum(1)
        m["d_row_w"][s] = (h.abs() * dh0m).sum(1)
        g["d_a"][s] = dgu @ W13
        g["d_w13"][e] = dgu.T @ A
        g["d_w2"][e] = D.T @ (h * w)
        # rounded operands: one bf16 rounding of dgu / row_w*h, and the fp32 error of dh0 (through dgum)
        m["d_a"][s] = dgu.abs() @ W13.abs()
        m["d_w13"][e] = dgu.abs().T @ A.abs()
        m["d_w2"][e] = D.abs().T @ (h * w).abs()
        g.setdefault("_fp32", {})[e] = (dgum @ W13.abs(), dgum.T @ A.abs())
    fp = g.pop("_fp32")
    f = dict(d_a=z(R, H), d_w13=z(E, 2 * I, H))
    for e in range(E):
        f["d_a"][offsets[e]:offsets[e + 1]], f["d_w13"][e] = fp[e]
    return g, m, f


def backward_tolerance(name, ref, mag, fp32mag, H, I, rows, out_dtype=torch.bfloat16):
    """Elementwise bound on a gradient's error.

    Output: one rounding (U_out |ref|). bf16 gradients' second operand (dg, du
    or row_w h) is rounded once: U_bf16 on every term, so U_bf16 * mag. Sums of
    n fp32 terms: at most n U_f32 per term of the sum's magnitudes. The
    sigmoid (exp and a fast division) is good to 2^-20 relative on every
    factor it enters, taken 4 times."""
    U_out = BF16_U if out_dtype == torch.bfloat16 else F32_U
    fast = 4 * 2.0 ** -20
    if name == "d_row_w":
        return F32_U * ref.abs() + ((H + I) * F32_U + fast) * mag
    n = {"d_a": 2 * I, "d_w13": rows, "d_w2": rows}[name]
    tol = U_out * ref.abs() * (1 + 2 * BF16_U) + (BF16_U + n * F32_U + fast) * mag
    if fp32mag is not None:
        tol = tol + H * F32_U * fp32mag
    return tol


def route_weights(logits, ids, scoring, norm, scale):
    """Routing weights [T, k] of the chosen experts, float64, differentiable in logits."""
    s = torch.softmax(logits, 1) if scoring == "softmax" else torch.sigmoid(logits)
    w = s.gather(1, ids.long())
    if norm:
        w = w / w.sum(1, keepdim=True)
    return w * scale
