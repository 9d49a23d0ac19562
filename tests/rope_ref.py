"""Rotary positions on the CPU in 64 bits, from their definition (include/rope.h)."""
import torch


def rotate(x, freqs, positions, amplitude=1.0, interleaved=False, transposed=False):
    """x [B, H, N, D], positions [B, N] or [N]: fp64 rows, pair by pair."""
    y = x.double().clone()
    pos = positions.double().expand(x.shape[0], x.shape[2])
    for i, f in enumerate(freqs):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + len(freqs))
        t = (pos * f)[:, None]
        c, s = amplitude * torch.cos(t), amplitude * torch.sin(t) * (-1.0 if transposed else 1.0)
        u, v = x[..., a].double(), x[..., b].double()
        y[..., a], y[..., b] = u * c - v * s, v * c + u * s
    return y


def partner(x, rot, interleaved):
    """|x| + |the other half of its pair| of the dimensions that turn, 0 of the others."""
    m = torch.zeros_like(x, dtype=torch.float64)
    r = x[..., :rot].double().abs()
    o = r.unflatten(-1, (rot // 2, 2)).flip(-1).flatten(-2) if interleaved else r.roll(rot // 2, -1)
    m[..., :rot] = r + o
    return m


# What the arithmetic adds to a result before it is rounded, relative to A (|a| + |b|): the angle
# is off by 2^-25 of half a turn (2^-23.3 radians), sine and cosine by 2 units of 2^-24 more, the
# amplitude and two products and their sum by 4 units of 2^-24.  Together under 2^-21.
ARITH = 2.0 ** -21


def tolerance(x, ref, dtype, rot, interleaved, amplitude):
    """How far a rotated row of x may be from ref: half a step of its type, and ARITH."""
    half = torch.finfo(dtype).eps / 2
    least = 2.0 ** -25 if dtype is torch.float16 else 2.0 ** -134   # half of the smallest subnormal
    return ref.abs() * half * (1 + 2.0 ** -10) + least + amplitude * partner(x, rot, interleaved) * ARITH * (1 + half)
