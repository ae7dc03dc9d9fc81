"""fp64 numpy oracle of the operators around the attention: residual and RMS
norm, 8-bit blocks and their product, rotary positions over three axes, each
with its gradient where the library has one.  Written from the formulas;
shares no code with the library."""
from __future__ import annotations

import math
from typing import Optional, Sequence, Tuple

import numpy as np

E4M3_MAX = 448.0
TINY = 2.0 ** -100


# ---------------------------------------------------------------- norm

def rms_norm(h: np.ndarray, w: np.ndarray, eps: float) -> Tuple[np.ndarray, np.ndarray]:
    """(y, rstd) of rows h [R, C]."""
    rstd = 1.0 / np.sqrt((h * h).mean(-1) + eps)
    return h * rstd[:, None] * w, rstd


def rms_norm_backward(h, w, eps, dy, dh=None):
    """(d, dw): gradient of h (from y and from h itself) and of the weight."""
    _, rstd = rms_norm(h, w, eps)
    r = rstd[:, None]
    g = dy * w
    d = r * (g - h * (g * h).mean(-1, keepdims=True) * r * r)
    return (d if dh is None else d + dh), (dy * h * r).sum(0)


# ---------------------------------------------------------------- 8 bits

def block_scales(y: np.ndarray) -> np.ndarray:
    """Scales [ceil(C/128), R] of rows y [R, C]."""
    R, C = y.shape
    return np.stack([np.maximum(np.abs(y[:, c:c + 128]).max(1), TINY) / E4M3_MAX for c in range(0, C, 128)]) \
        if R else np.zeros((-(-C // 128), 0))


def spread(scale: np.ndarray, C: int) -> np.ndarray:
    """Row scales [blocks, R] as one factor per element [R, C]."""
    return np.repeat(scale.T, 128, 1)[:, :C]


def spread_weight(scale: np.ndarray, N: int, K: int) -> np.ndarray:
    return np.repeat(np.repeat(scale, 128, 0), 128, 1)[:N, :K]


# ---------------------------------------------------------------- rotary positions

def pairs(dims: Sequence[int], halves: bool):
    """(first channel, second channel, axis, index in the axis) of each turned pair."""
    out, at = [], 0
    for axis, dim in enumerate(dims):
        for i in range(dim // 2):
            out.append((at + i, at + dim // 2 + i, axis, i) if halves else (at + 2 * i, at + 2 * i + 1, axis, i))
        at += dim
    return out


def turn(x: np.ndarray, grid, dims, tables, halves: bool, sign: float = 1.0) -> np.ndarray:
    """x [B, N, heads, d] with its pairs turned by their tokens' angles (sign -1: back)."""
    T, H, W = grid
    n = np.arange(T * H * W)
    place = (n // (H * W), n // W % H, n % W)
    y = x.copy()
    for a, b, axis, i in pairs(dims, halves):
        c = tables[axis][place[axis], i, 0][None, :, None]
        s = sign * tables[axis][place[axis], i, 1][None, :, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def _mean(x, norm):
    return x.mean((-1, -2), keepdims=True) if norm == "row" else x.mean(-1, keepdims=True)


def norm_rope(x, w: Optional[np.ndarray], grid, dims, tables, norm, halves, eps):
    """[B, N, heads, d] -> grid order [B, heads, N, d]."""
    if norm != "none":
        x = x / np.sqrt(_mean(x * x, norm) + eps) * w.reshape(-1, x.shape[-1])
    return turn(x, grid, dims, tables, halves).transpose(0, 2, 1, 3)


def norm_rope_backward(x, w, grid, dims, tables, norm, halves, eps, dout):
    """(dx, dw, |terms| of dx, |terms| of dw): gradients for dout [B, heads, N, d], and the sums of the
    magnitudes that were added up for each of them (what a rounding error of fp32 sums is relative to)."""
    dt = dout.transpose(0, 2, 1, 3)
    g = turn(dt, grid, dims, tables, halves, -1.0)
    gm = np.abs(dt)
    swap = gm.copy()
    for a, b, _, _ in pairs(dims, halves):
        swap[..., a] = swap[..., b] = gm[..., a] + gm[..., b]
    if norm == "none":
        return g, None, swap, None
    r = 1.0 / np.sqrt(_mean(x * x, norm) + eps)
    wf = np.broadcast_to(w.reshape(-1, x.shape[-1]), x.shape[2:])
    dx = r * (g * wf - x * _mean(g * wf * x, norm) * r * r)
    mag = r * (swap * np.abs(wf) + np.abs(x) * _mean(swap * np.abs(wf * x), norm) * r * r)
    axes = (0, 1) if norm == "row" else (0, 1, 2)
    return dx, (g * x * r).sum(axes).reshape(-1), mag, (swap * np.abs(x) * r).sum(axes).reshape(-1)


def rope_table(n: int, dim: int, theta: float, start: float, step: float) -> np.ndarray:
    """(cos, sin) [n, dim/2, 2]."""
    out = np.empty((n, dim // 2, 2))
    for i in range(n):
        for j in range(dim // 2):
            a = (start + step * i) * theta ** (-2.0 * j / dim)
            out[i, j] = math.cos(a), math.sin(a)
    return out
