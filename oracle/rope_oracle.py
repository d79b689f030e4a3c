"""FP64 CPU oracle for the norms of the q and k heads with the position rotation (test infrastructure).

TEST INFRASTRUCTURE ONLY, as the other oracles: the product path never imports it, and it imports
nothing from the product. Per head row x [d] at position p, weight w or ones:

    n = x / sqrt(mean(x^2) + eps)  ("rms"),  x / sqrt(sum(x^2) + eps)  ("l2"),  x  ("none")
    z = n w;  y = z with the pairs (a, b) of its first rotary_dim values turned by p f_i and scaled by m:
    y_a + i y_b = m (z_a + i z_b) exp(i p f_i)
    pairs (i, i + rotary_dim / 2), or (2 i, 2 i + 1) when interleaved

Backward for an upstream gradient dy: dz_a + i dz_b = m (dy_a + i dy_b) exp(-i p f_i); dn = dz w;
dw = sum over rows of dz n; dx = r (dn - c n (n . dn)) with r the factor of x in n, c = 1/d ("rms"),
1 ("l2"); dx = dz ("none").
"""
from __future__ import annotations

import math

import numpy as np


def frequencies(rotary_dim, base=10000.0, scaling="none", factor=1.0, original_length=0.0, fast=32.0, slow=1.0):
    """(f [rotary_dim / 2] in radians per position, magnitude)."""
    i = np.arange(rotary_dim // 2)
    if scaling == "ntk":
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    f = base ** (-2.0 * i / rotary_dim)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling in ("yarn", "bands"):
        if scaling == "yarn":
            at = lambda turns: rotary_dim * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(base))
            lo, hi = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), rotary_dim - 1)
            r = (i - lo) / max(hi - lo, 0.001)
        else:
            r = 1 - (original_length * f / (2 * math.pi) - slow) / (fast - slow)
        r = np.clip(r, 0, 1)
        return f * (1 - r) + f / factor * r, 0.1 * math.log(factor) + 1 if scaling == "yarn" and factor > 1 else 1.0
    return f, 1.0


def _turn(z, angle, rotary_dim, interleaved, m):
    """z [T, h, d] with its pairs multiplied by m exp(i angle), angle [T, rotary_dim / 2]."""
    out = z.copy()
    r = rotary_dim
    a, b = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    w = (z[..., a] + 1j * z[..., b]) * (m * np.exp(1j * angle))[:, None, :]
    out[..., a], out[..., b] = w.real, w.imag
    return out


def _factor(x, norm, eps):
    """(r, c): n = x r, and the c of the backward."""
    if norm == "rms":
        return 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps), 1 / x.shape[-1]
    if norm == "l2":
        return 1 / np.sqrt(np.sum(x * x, -1, keepdims=True) + eps), 1.0
    return np.ones(x.shape[:-1] + (1,)), 0.0


def fwd(x, positions, f, w=None, norm="rms", rotary_dim=None, interleaved=False, eps=1e-6, m=1.0):
    """y [T, h, d] of x [T, h, d]."""
    x = np.asarray(x, dtype=np.float64)
    r, _ = _factor(x, norm, eps)
    z = x * r if w is None else x * r * np.asarray(w, dtype=np.float64)
    angle = np.asarray(positions, dtype=np.float64)[:, None] * f
    return _turn(z, angle, x.shape[-1] if rotary_dim is None else rotary_dim, interleaved, m)


def bwd(x, dy, positions, f, w=None, norm="rms", rotary_dim=None, interleaved=False, eps=1e-6, m=1.0):
    """(dx [T, h, d], dw [d] or None)."""
    x, dy = np.asarray(x, dtype=np.float64), np.asarray(dy, dtype=np.float64)
    r, c = _factor(x, norm, eps)
    n = x * r
    angle = np.asarray(positions, dtype=np.float64)[:, None] * f
    dz = _turn(dy, -angle, x.shape[-1] if rotary_dim is None else rotary_dim, interleaved, m)
    dn = dz if w is None else dz * np.asarray(w, dtype=np.float64)
    dx = r * (dn - c * n * np.sum(n * dn, -1, keepdims=True))
    return dx, None if w is None else np.sum(dz * n, axis=(0, 1))
