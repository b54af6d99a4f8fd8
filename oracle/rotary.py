"""Rotary positions with the norm of each head's vector, in 64 bits, from the definition."""
from __future__ import annotations

import math

import numpy as np

DIM = 256


def frequency(i: int, rotary_dim: int, base: float, scaling: str = "none", factor: float = 1.0, original: float = 0.0,
              low: float = 0.0, high: float = 0.0) -> float:
    """Radians per position of pair i."""
    n = rotary_dim // 2
    if scaling == "ntk":
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    f = base ** (-i / n)
    if scaling == "linear":
        return f / factor
    if scaling == "yarn":
        # pair number x turns original / (2 pi) * base^(-x/n) times within the original length
        begin = max(0.0, math.floor(n * math.log(original / (2 * math.pi * high), base)))
        end = min(rotary_dim - 1.0, math.ceil(n * math.log(original / (2 * math.pi * low), base)))
        stretched = min(1.0, max(0.0, (i - begin) / (end - begin if end > begin else 0.001)))
        return (1 - stretched) * f + stretched * f / factor
    if scaling == "banded":
        turns = original * f / (2 * math.pi)
        if turns >= high:
            return f
        if turns <= low:
            return f / factor
        return f / factor + (f - f / factor) * (turns - low) / (high - low)
    return f


def norm(x: np.ndarray, weight: np.ndarray, eps: float) -> np.ndarray:
    x = np.asarray(x, dtype=np.float64)
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight


def turn(x: np.ndarray, positions: np.ndarray, frequencies, interleaved: bool, amplitude: float = 1.0) -> np.ndarray:
    """x [..., rows, 256]; positions [..., rows], broadcast against x's leading dims: as complex numbers a + ib times amplitude * e^(i angle)."""
    n = len(frequencies)
    out = np.array(x, dtype=np.float64)
    a = slice(0, 2 * n, 2) if interleaved else slice(0, n)
    b = slice(1, 2 * n, 2) if interleaved else slice(n, 2 * n)
    angle = np.asarray(positions, dtype=np.longdouble)[..., None] * np.asarray(frequencies, dtype=np.longdouble)
    angle = np.remainder(angle, 2 * np.longdouble(np.pi)).astype(np.float64)
    z = (out[..., a] + 1j * out[..., b]) * (amplitude * np.exp(1j * angle))
    out[..., a], out[..., b] = z.real, z.imag
    return out
