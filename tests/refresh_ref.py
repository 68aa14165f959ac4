"""64-bit statements of the refresh operators (norm + rotation, 4-bit cache, attention over it),
for the tests: plain torch on the tensors' device, no code of the library."""
import math

import torch


def frequencies(R, base, factor=1.0, bands=None):
    """bands: (original_len, slow_turns, fast_turns) or None for linear scaling."""
    f = []
    for i in range(R // 2):
        g = base ** (-2.0 * i / R)
        if bands is None:
            f.append(g / factor)
        else:
            turns = bands[0] * g / (2 * math.pi)
            w = min(1.0, max(0.0, (turns - bands[1]) / (bands[2] - bands[1])))
            f.append((1 - w) * g / factor + w * g)
    return torch.tensor(f, dtype=torch.float64)


def norm_rope(x, pos, freq, weight, eps, interleaved, magnitude=1.0, norm=True):
    """x [B, n, H, D]; pos [B, n]; freq [R / 2] float64 or None. Also returns the norm of each
    channel's pair (the scale of its rounding error)."""
    y = x.double()
    if norm:
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + eps)
        if weight is not None:
            y = y * weight.double()
    size = y.abs().clone()
    if freq is not None:
        R = 2 * freq.numel()
        i = torch.arange(R // 2, device=x.device)
        ia, ic = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        t = (pos.double()[:, :, None] * freq.to(x.device))[:, :, None, :]
        a, c = y[..., ia].clone(), y[..., ic].clone()
        y[..., ia] = (a * torch.cos(t) - c * torch.sin(t)) * magnitude
        y[..., ic] = (c * torch.cos(t) + a * torch.sin(t)) * magnitude
        pair = torch.hypot(a, c) * abs(magnitude)
        size[..., ia] = pair
        size[..., ic] = pair
    return y, size


def steps(x):
    """Step and zero point of each group of 32 of x [..., D] (float64)."""
    g = x.double().unflatten(-1, (-1, 32))
    lo, hi = g.amin(-1).clamp(max=0), g.amax(-1).clamp(min=0)
    s0 = (hi - lo) / 15
    e = torch.floor(torch.log2(torch.where(s0 > 0, s0, torch.ones_like(s0))))
    unit = torch.exp2(e - 2)  # three significant bits
    s = torch.ceil(s0 / unit) * unit
    s = torch.where(s0 < 2.0 ** -110, torch.zeros_like(s), s)
    z = torch.floor(-lo / torch.where(s > 0, s, torch.ones_like(s)) + 0.5)
    return s, z


def quantised(x):
    """Values [..., D] (float64) that x [..., D] reads back as."""
    s, z = steps(x)
    s, z = s.unsqueeze(-1), z.unsqueeze(-1)
    g = x.double().unflatten(-1, (-1, 32))
    r = g / torch.where(s > 0, s, torch.ones_like(s))
    near = torch.sign(r) * torch.floor(r.abs() + 0.5)
    n = (near + z).clamp(0, 15)
    return ((n - z) * s).flatten(-2)


def unpack(codes, params):
    """Codes and params tensors -> values [..., D] (float64), from the documented format."""
    c = codes.long()
    n = torch.stack((c % 16, c // 16), -1).flatten(-2).unflatten(-1, (-1, 32))
    w = params.long() % 65536
    s = ((w - w % 32) * 65536).to(torch.int32).view(torch.float32).double()
    return ((n - (w % 16).unsqueeze(-1)).double() * s.unsqueeze(-1)).flatten(-2)


def attention(q, k, v, seen, scale):
    """q [B, n, Hq, D]; k, v [B, T, Hkv, D]; seen [B, n, T] bool.  Returns out, lse and, per
    output, sum_j p_j |v_j| and the largest sum_c |q_c k_c| (scales of the rounding errors)."""
    B, n, Hq, D = q.shape
    G = Hq // k.shape[2]
    kk, vv = (x.double().repeat_interleave(G, 2).permute(0, 2, 1, 3) for x in (k, v))
    hidden = ~seen.any(1)[:, None, :, None]  # entries no query sees may hold anything
    kk, vv = kk.masked_fill(hidden, 0.0), vv.masked_fill(hidden, 0.0)
    qq = q.double().permute(0, 2, 1, 3)
    s = (qq @ kk.transpose(2, 3)) * scale
    s = s.masked_fill(~seen[:, None], -math.inf)
    lse = torch.logsumexp(s, -1) if s.shape[-1] else torch.full((B, Hq, n), -math.inf, device=q.device).double()
    p = torch.exp(s - torch.where(lse > -math.inf, lse, torch.zeros_like(lse))[..., None])
    out, mag = p @ vv, p @ vv.abs()
    prod = (qq.abs() @ kk.abs().transpose(2, 3)) * abs(scale)
    top = prod.amax(-1) if s.shape[-1] else torch.zeros_like(lse)
    return out.permute(0, 2, 1, 3), lse, mag.permute(0, 2, 1, 3), top
