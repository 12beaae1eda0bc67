"""Oracle: the decoder block's parts around the experts, straight from their definitions in float64.

TEST INFRASTRUCTURE, like the rest of this package: plain numpy, row by row, nothing shared with the CUDA path.

  norm       h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight
  attention  softmax(scale * q k^T) v over the keys a row sees: key j for the row at position p when j <= p and
             (no window, or p - j < window, or j < sinks)
"""
from __future__ import annotations

import numpy as np

from . import formats as F


def add_rmsnorm(x, residual, weight, eps):
    """(h, y) in float64, unrounded."""
    h = np.asarray(x, dtype=np.float64)
    if residual is not None:
        h = h + np.asarray(residual, dtype=np.float64)
    y = h / np.sqrt(np.mean(h * h, axis=-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)
    return h, y


def visible(p: int, n: int, window: int, sinks: int) -> np.ndarray:
    """The indexes of the keys among n that the row at position p sees."""
    return np.array([j for j in range(min(n, p + 1)) if not window or p - j < window or j < sinks], dtype=np.int64)


def attend(q, k, v, p0: int, scale: float, window: int = 0, sinks: int = 0):
    """Rows q [R, D] at positions p0, p0 + 1, ... over k, v [n, D]. Returns (out, mag): the result and the weighted sum
    of the values' magnitudes, which bounds its rounding errors. Keys that a row does not see are not touched."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    out = np.zeros((q.shape[0], v.shape[1]))
    mag = np.zeros_like(out)
    for r in range(q.shape[0]):
        see = visible(p0 + r, k.shape[0], window, sinks)
        if not len(see):
            continue
        s = k[see] @ q[r] * scale
        w = np.exp(s - np.max(s))
        w /= w.sum()
        out[r], mag[r] = w @ v[see], w @ np.abs(v[see])
    return out, mag


def attend_heads(q, k, v, p0, scale, window=0, sinks=0):
    """q [R, Hq, D], k and v [n, Hkv, D]: head h of q reads head h // (Hq / Hkv)."""
    group = q.shape[1] // k.shape[1]
    both = [attend(q[:, h], k[:, h // group], v[:, h // group], p0, scale, window, sinks) for h in range(q.shape[1])]
    return np.stack([o for o, _ in both], 1), np.stack([m for _, m in both], 1)


def attention_tolerance(out, mag):
    """How far a kernel may be that rounds its softmax weights to bf16 and its result once more.

    A rounding to bf16 is off by at most 2^-8 of the value. If every weight were
    off by the most, in the weighted sum one way and in the sum that it is divided by the other, that would make 2^-7 of
    the weighted magnitudes, and 2^-8 of the result for its own rounding. Half of either is asked for, because weights
    round both ways (a row with few of them has to do better than one rounding each). fp32 scores and sums add less than
    2^-10 at the tested sizes (a score is a sum of 128 products, off by less than 128 * 2^-24 of their magnitudes, which
    stay below 50)."""
    return (2.0 ** -8 + 2.0 ** -10) * mag + 2.0 ** -9 * np.abs(out) + 1e-30


def quant_block_mxfp8(x):
    """The cache's MXFP8 rule for rows [..., D]: (codes, scales) as uint8; a block with a value that is not finite has
    scale byte 255."""
    from . import moe as M
    x = np.asarray(x, dtype=np.float32)
    rows = x.reshape(-1, x.shape[-1])
    fine = np.isfinite(rows.reshape(rows.shape[0], -1, F.BLOCK)).all(-1)
    safe = np.where(np.repeat(fine, F.BLOCK, axis=1), rows, 0)
    q, s = M.quant_mxfp8(safe)
    s = np.where(fine, s, 255).astype(np.uint8)
    return q.reshape(x.shape), s.reshape(*x.shape[:-1], -1)


def quant_block_mxfp4(x):
    """The cache's MXFP4 rule for rows [..., D]: (codes two to a byte [..., D/2], scales) as uint8; a block with a value that
    is not finite has codes of zero and scale byte 255."""
    from . import moe as M
    x = np.asarray(x, dtype=np.float32)
    rows = x.reshape(-1, x.shape[-1])
    fine = np.isfinite(rows.reshape(rows.shape[0], -1, F.BLOCK)).all(-1)
    q, s = M.quant_mxfp4(np.where(np.repeat(fine, F.BLOCK, axis=1), rows, 0))
    s = np.where(fine, s, 255).astype(np.uint8)
    return q.reshape(*x.shape[:-1], -1), s.reshape(*x.shape[:-1], -1)


def rope(x, pos, inv_freq, axis=None, interleaved=False, factor=1.0, inverse=False):
    """Rows x [T, heads, D] turned by their positions pos [axes, T], pair by pair. Returns (out, mag): the result, and
    |a| + |b| of the pair times the factor, which bounds the rounding of its two products."""
    x = np.asarray(x, dtype=np.float64)
    out, mag = x.copy(), np.zeros_like(x)
    half = len(inv_freq)
    for i, w in enumerate(np.asarray(inv_freq, dtype=np.float64)):
        t = np.asarray(pos[axis[i] if axis is not None else 0], dtype=np.float64) * w * (-1 if inverse else 1)
        i0, i1 = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        a, b = x[..., i0], x[..., i1]
        c, s = factor * np.cos(t)[:, None], factor * np.sin(t)[:, None]
        out[..., i0], out[..., i1] = a * c - b * s, a * s + b * c
        mag[..., i0] = mag[..., i1] = abs(factor) * (np.abs(a) + np.abs(b))
    return out, mag
