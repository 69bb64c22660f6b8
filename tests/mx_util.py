"""MXFP4 in float64 torch (not a test module): E2M1 values, one power-of-two
scale per 32, from the format's definition."""
import torch

F64 = torch.float64
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def scale_bytes(v):
    """[.., K] -> [.., K/32] int64 scale bytes."""
    b = v.to(F64).reshape(*v.shape[:-1], -1, 32)
    amax = torch.where(torch.isnan(b), torch.full_like(b, float("inf")), b.abs()).amax(-1)
    e = torch.frexp(amax)[1].long() - 1 - 2
    s = e.clamp(-127, 125) + 127
    s = torch.where(amax == 0, torch.full_like(s, 127), s)
    return torch.where(torch.isinf(amax), torch.full_like(s, 255), s)


def pow2(e):
    """2^e exactly, for e in [-1000, 1000]."""
    return ((e.long() + 1023) << 52).view(F64)


def quantize(v):
    """[.., K] -> (codes [.., K] int64 0..15, scale bytes [.., K/32])."""
    s = scale_bytes(v)
    b = v.to(F64).reshape(*v.shape[:-1], -1, 32)
    unit = pow2(torch.where(s == 255, torch.zeros_like(s), s - 127))
    a = (b.abs() / unit.unsqueeze(-1)).nan_to_num(nan=7.0, posinf=7.0)
    grid = torch.tensor(GRID, dtype=F64, device=v.device)
    dist = (a.unsqueeze(-1) - grid).abs()
    best = dist.amin(-1, keepdim=True)
    tie = dist == best
    idx = torch.arange(8, device=v.device).expand_as(tie)
    even = torch.where(tie, idx + 100 * (idx % 2), torch.full_like(idx, 1000)).argmin(-1)
    code = even + 8 * torch.signbit(b).long()
    return code.reshape(v.shape), s


def values(code, s):
    """The float64 values of codes [.., K] with scale bytes [.., K/32]."""
    grid = torch.tensor(GRID + [-g for g in GRID], dtype=F64, device=code.device)
    u = torch.where(s == 255, torch.full(s.shape, float("nan"), dtype=F64, device=s.device),
                    pow2(torch.where(s == 255, torch.zeros_like(s), s - 127)))
    return (grid[code].reshape(*s.shape, 32) * u.unsqueeze(-1)).reshape(code.shape)


def pack(code):
    return (code[..., 0::2] | (code[..., 1::2] << 4)).to(torch.uint8)


def unpack(q):
    q = q.long()
    return torch.stack([q & 15, q >> 4], -1).reshape(*q.shape[:-1], -1)


def row_scale_words(s):
    """Scale bytes [R, K/32] as the kernels' [K/128, R, 4]."""
    return s.reshape(s.shape[0], -1, 4).transpose(0, 1).contiguous().to(torch.uint8)


def weight_scale_blocks(s):
    """Scale bytes [E, N, K/32] as the kernels' [E, N/128, K/128, 512]."""
    E, N, S = s.shape
    out = torch.empty(E, N // 128, S // 4, 512, dtype=torch.uint8, device=s.device)
    for r in range(128):
        for j in range(4):
            out[..., (r % 32) * 16 + (r // 32) * 4 + j] = s.reshape(E, N // 128, 128, S // 4, 4)[:, :, r, :, j].to(torch.uint8)
    return out


def half_step(a):
    """Largest distance from |v| / scale = a to its code's value (a < 8)."""
    return torch.where(a <= 2, 0.25, torch.where(a <= 4, 0.5, torch.where(a <= 6, 1.0, a - 6 + 1e-30)))
