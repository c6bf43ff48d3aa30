"""Plain 64-bit definitions of the layer operators, on the CPU: what the tests
of moe_norm, moe_linear, moe_kv_append and moe_kv_attend compare with."""
import math

import torch

PAGE = 64
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def e4m3(codes):
    """Values of E4M3 codes (uint8), float64; 0x7F and 0xFF are NaN."""
    c = codes.long()
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e.double() - 10))
    v = torch.where((c & 127) == 127, math.nan, v)
    return torch.where(c >= 128, -v, v)


def to_e4m3(v):
    """Nearest E4M3 value, ties to even (|v| <= 448)."""
    step = 2.0 ** (torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def half_step(v):
    """Half the distance of E4M3 values around v."""
    return 2.0 ** (torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 4)


def pow2_scale(amax):
    """Smallest power of two s >= 2^-64 with amax <= 448 s."""
    out = []
    for a in amax.reshape(-1).tolist():
        e = -64
        while a > 448 * 2.0 ** e:
            e += 1
        out.append(2.0 ** e)
    return torch.tensor(out, dtype=torch.float64).reshape(amax.shape)


def norm(x, r, w, eps):
    s = x.double() + (0 if r is None else r.double())
    return s, s / torch.sqrt((s * s).mean(-1, keepdim=True) + eps) * w.double()


def nvfp4(q, s):
    lut = torch.tensor(_E2M1 + [-v for v in _E2M1], dtype=torch.float64)
    w = torch.stack((lut[(q & 15).long()], lut[(q >> 4).long()]), -1).flatten(-2)
    return w * e4m3(s).repeat_interleave(16, dim=-1)


def rotate(x, rope, interleaved):
    """x float64 [n, heads, D], rope [n, R] of (cos, sin)."""
    R = rope.shape[1]
    y = x.clone()
    for j in range(R // 2):
        i0, i1 = (2 * j, 2 * j + 1) if interleaved else (j, j + R // 2)
        c, s = rope[:, 2 * j, None].double(), rope[:, 2 * j + 1, None].double()
        y[..., i0], y[..., i1] = x[..., i0] * c - x[..., i1] * s, x[..., i1] * c + x[..., i0] * s
    return y


def attend(q, k, v, n, L, scale):
    """One sequence, one kv head: q [n, G, D], k and v [L, D] -> o [n, G, D], the
    sum of |weight * v|, the normalised sum over the largest weight, and the
    largest visible |v| of each row."""
    G, D = q.shape[1:]
    o = torch.zeros((n, G, D), dtype=torch.float64)
    A = torch.zeros((n, G, D), dtype=torch.float64)
    ln = torch.ones((n, G), dtype=torch.float64)
    vm = torch.zeros((n, G), dtype=torch.float64)
    for i in range(n):
        m = min(max(L - n + i + 1, 0), L)
        if m == 0:
            continue
        s = (q[i].double() @ k[:m].T) * scale
        p = torch.exp(s - s.amax(-1, keepdim=True))
        ln[i] = p.sum(-1)
        p = p / p.sum(-1, keepdim=True)
        o[i] = p @ v[:m]
        A[i] = p @ v[:m].abs()
        vm[i] = v[:m].abs().max()
    return o, A, ln, vm
