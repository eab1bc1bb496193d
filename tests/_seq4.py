"""Shared by the tests of the 4-bit cache and of appending with the rotation: the cache's grid and plain forms."""
import math

import torch


def scale_of(byte):
    """What a scale's byte stands for, in 64 bits: (1 + m / 8) 2^(e - 15), NaN from e = 31 on."""
    unit = [(8 + i % 8) * 2.0 ** (i // 8 - 18) if i < 248 else math.nan for i in range(256)]
    return torch.tensor(unit, dtype=torch.float64, device=byte.device)[byte.long()]


def quantise4(x):
    """Bytes [..., d / 2], scale bytes [..., d / 32] and the values they stand for (64 bits) of x [..., d] in 32 bits or fewer. The
    scale is the nearest of the grid to the 32-bit quotient amax / 7, a code the nearest whole number to the 32-bit quotient
    x / scale (IEEE quotients of tensors; ties to even both)."""
    g = x.float().unflatten(-1, (-1, 32))
    bad = ~torch.isfinite(g).all(-1, keepdim=True)
    top = torch.where(bad, torch.zeros_like(g[..., :1]), g.abs().amax(-1, keepdim=True))
    want = (top / torch.full_like(top, 7.0)).double()
    grid = scale_of(torch.arange(8, 248, device=x.device))
    above = torch.searchsorted(grid, want).clamp(1, len(grid) - 1)
    low, high = grid[above - 1], grid[above]
    up = (high - want < want - low) | ((high - want == want - low) & (above % 2 == 0))
    at = torch.where(up, above, above - 1)
    unit = grid[at]
    code = torch.round((torch.where(bad, torch.zeros_like(g), g) / unit.float()).double()).clamp(-7, 7)
    byte = torch.where(bad, torch.full_like(at, 255), at + 8).to(torch.uint8)[..., 0]
    val = torch.where(bad, torch.full_like(code, math.nan), code * unit).flatten(-2)
    code = (code + 8).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), byte, val


def values4(byte, scale):
    """The values of a 4-bit cache's bytes in 64 bits."""
    x = torch.stack([byte & 15, byte >> 4], -1).flatten(-2).double() - 8
    return (x.unflatten(-1, (-1, 32)) * scale_of(scale)[..., None]).flatten(-2)


def turned(x, cos_sin, position, interleaved):
    """x [T, heads, d] with its first rot features' pairs turned, in 32 bits, a rounded product and sum at a time."""
    rot = cos_sin.shape[1]
    half, x = rot // 2, x.float()
    c, s = cos_sin[position][:, None, :half], cos_sin[position][:, None, half:]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :half], x[..., half:rot])
    ac, bs, bc, as_ = a * c, b * s, b * c, a * s
    y = x.clone()
    if interleaved:
        y[..., 0:rot:2], y[..., 1:rot:2] = ac - bs, bc + as_
    else:
        y[..., :half], y[..., half:rot] = ac - bs, bc + as_
    return y
