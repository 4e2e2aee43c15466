"""Plain 64-bit forms of the operators around a layer's state, on the CPU, straight from their formulas."""
from __future__ import annotations

import math

import torch

from serve_ref import f64

E4M3 = torch.float8_e4m3fn


def norm(x, weight, residual=None, eps=1e-6):
    """(y, h), both like x."""
    h = f64(x) if residual is None else f64(x) + f64(residual)
    y = h / torch.sqrt(h.square().mean(-1, keepdim=True) + eps)
    return y if weight is None else y * f64(weight), h


def groups(x, rows):
    """x [n, K] as [blocks, rows, blocks, 128], zeros behind the end."""
    n, K = x.shape
    return torch.nn.functional.pad(x, (0, -K % 128, 0, -n % rows)).unflatten(1, (-1, 128)).unflatten(0, (-1, rows))


def quantize(x, rows):
    """8-bit values and scales in fp32 steps: the rounding is part of the definition."""
    x = x.detach().cpu().float()
    g = groups(x, rows)
    top = torch.where(g.isnan().any(3).any(1), torch.full((), math.nan), g.abs().amax((1, 3)))
    scale = top * torch.tensor(1.0 / 448.0, dtype=torch.float32)
    scale = torch.where(scale < 2.0 ** -126, torch.full((), 2.0 ** -126), scale)
    y = g * (torch.ones(()) / scale)[:, None, :, None]
    y = torch.where(y.isnan(), y, y.clamp(-448, 448))
    return y.flatten(0, 1).flatten(1)[:x.shape[0], :x.shape[1]].to(E4M3), scale


def wide(y, scale, rows):
    """The values that 8-bit ones stand for, in 64 bits."""
    n, K = y.shape
    return y.detach().cpu().float().double() * f64(scale).repeat_interleave(rows, 0)[:n].repeat_interleave(128, 1)[:, :K]


def matmul(x, xs, w, ws):
    """(o, sum of the terms' magnitudes)."""
    a, b = wide(x, xs, 1), wide(w, ws, 128)
    return a @ b.t(), a.abs() @ b.abs().t()


def rotary(x, positions, freq, interleaved, scale):
    """(x turned, |u| + |v| of each value's pair)."""
    x, half = f64(x), freq.shape[0]
    pos = positions.cpu().double()
    turns = pos[:, None] * (f64(freq) / (2 * math.pi))
    a = 2 * math.pi * (turns - turns.round())
    c, s = (torch.cos(a) * scale)[:, None], (torch.sin(a) * scale)[:, None]
    part = x[..., :2 * half]
    u, v = (part[..., 0::2], part[..., 1::2]) if interleaved else (part[..., :half], part[..., half:])
    join = (lambda p, q: torch.stack([p, q], -1).flatten(-2)) if interleaved else (lambda p, q: torch.cat([p, q], -1))
    still = (pos < 0)[:, None, None]
    o, size = x.clone(), torch.zeros_like(x)
    o[..., :2 * half] = torch.where(still, part, join(u * c - v * s, v * c + u * s))
    size[..., :2 * half] = torch.where(still, torch.zeros_like(part), join(u.abs() + v.abs(), u.abs() + v.abs()) * abs(scale))
    return o, size
