"""The 4-bit cache format in 64 bits, from its definition by search, and error bounds of attention
over it."""
import math

import torch

F64 = torch.float64
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def scale_of(byte):
    """f16 numbers of three mantissa bits: multiples of 2^-17 up to 2^-14, then eight a binade."""
    b = byte.to(torch.int64)
    s = torch.where(b < 8, b.to(F64) * 2.0 ** -17, (8 + b % 8).to(F64) * torch.exp2((b // 8).to(F64) - 18))
    return torch.where(b > 226, torch.full_like(s, math.nan), s)


def quantise(x):
    """Values (float64, on the grid) of codes and scale bytes of rows [..., D]."""
    y = x.to(F64).unflatten(-1, (-1, 16))
    bad = ~torch.isfinite(y).all(-1)
    y = torch.where(bad[..., None], torch.zeros_like(y), y)
    all_scales = scale_of(torch.arange(227, device=x.device))
    byte = torch.searchsorted(6 * all_scales, y.abs().amax(-1)).clamp(max=226)     # the smallest that holds it
    s = all_scales[byte][..., None]
    z = torch.where(s > 0, y.abs() / s, torch.zeros_like(y))
    grid = torch.tensor(GRID, dtype=F64, device=x.device)
    hi = torch.searchsorted(grid, z.contiguous()).clamp(1, 7)
    up, down = grid[hi] - z, z - grid[hi - 1]
    at = torch.where((down < up) | ((down == up) & (hi % 2 == 1)), hi - 1, hi)     # ties to the even code
    value = torch.copysign(grid[at], y)
    byte = torch.where(bad, torch.full_like(byte, 255), byte)
    return value.flatten(-2), byte.to(torch.uint8)


def pack(value):
    """Codes of grid values, two a byte, the even element low."""
    grid = torch.tensor(GRID, dtype=F64, device=value.device)
    code = torch.searchsorted(grid, value.abs().contiguous()) + 8 * (value < 0)
    return (code[..., 0::2] | code[..., 1::2] << 4).to(torch.uint8)


def unpack(codes):
    """Grid values of codes."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).to(torch.int64)
    grid = torch.tensor(GRID, dtype=F64, device=codes.device)
    return torch.where(c >= 8, -grid[c % 8], grid[c % 8])


def values(codes, byte):
    """What cached rows stand for, float64."""
    return unpack(codes) * scale_of(byte).repeat_interleave(16, -1)


def bounds(out, weight, sums, D, dtype, softcap, keys, q_max, k_max, v_max, many):
    """What out and lse may be off by, from the formats alone.

    A score: D products added in 32 bits, each addition within 2^-23 (it may truncate); bf16 rows of q
    are exact in f16 but for elements below 2^-32 of the row's largest, which are off by 2^-40 of that;
    the cap adds 2^-21 of it.  A weight e^(s - m): the score's error twice (s and m), 2^-21 of the
    exponential and 2^-22 of its argument; then one rounding to f16, half a unit, or half of f16's
    smallest number, 2^-25, beside a largest weight of 2^7 at least; or, for many rows, to the handle's
    type (`many`).  The result: one rounding."""
    half = torch.finfo(dtype).eps / 2
    f16 = half if many else 2.0 ** -11
    score = (D + 4) * 2.0 ** -23 * sums + (softcap or 0.0) * 2.0 ** -21 + D * 2.0 ** -40 * q_max * k_max
    top = torch.clamp(sums, max=softcap) if softcap else sums
    p = 2 * score + 2.0 ** -21 + 2.0 ** -22 * top
    tiny = 2.0 ** -24 if dtype == torch.float16 else 2.0 ** -120
    tol_out = half * out.abs() + (f16 * (1 + 2.0 ** -7) + p)[..., None] * weight + keys * 2.0 ** -31 * v_max + tiny
    return tol_out, score + p + 2.0 ** -21
