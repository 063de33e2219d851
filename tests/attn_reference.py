"""The attention side's operators from their definitions, on the CPU in 64 bits (no code shared with the library).

Quantisers follow the header's rules: each quotient and product is a single-precision operation (numpy float32),
each rounding goes to the nearest grid value, ties to the even code, saturating.
"""
import math

import numpy as np
import torch

U24 = 2.0 ** -24  # half a step of fp32, relative

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1])


def nearest(x, grid):
    """Index of the grid value nearest to x >= 0 (float64), ties to the even index, the last beyond it."""
    x = np.asarray(x, np.float64)
    up = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    below, above = x - grid[up - 1], grid[up] - x
    even = np.where(up % 2 == 0, up, up - 1)
    return np.where(below < above, up - 1, np.where(above < below, up, even))


def stored(x, fmt, scale=1.0):
    """float64 values that a cache of format 0 (bf16), 1 (e4m3) or 2 (nvfp4) holds for x, a float32 array [..., d]."""
    x = np.asarray(x, np.float32)
    if fmt == 0:
        return torch.from_numpy(x).to(torch.bfloat16).double().numpy()
    if fmt == 1:
        amax = np.abs(x).max(-1, keepdims=True).astype(np.float64)
        with np.errstate(all="ignore"):
            m, e = np.frexp(amax)                      # amax = m 2^e, m in [0.5, 1)
        e = np.maximum(np.where(amax > 0, e - 9 + (m > 0.875), -110), -110)
        size = np.ldexp(1.0, np.where(np.isfinite(amax), e, 0))
        with np.errstate(invalid="ignore"):
            v = np.copysign(E4M3[nearest(np.abs(x.astype(np.float64)) / size, E4M3)] * size, x)
        return np.where(np.isfinite(amax), v, np.nan)
    st = np.float32(scale)
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    amax = np.abs(b).max(-1, keepdims=True)
    with np.errstate(all="ignore"):
        si = nearest(np.minimum(amax / (np.float32(6) * st), np.float32(448)), E4M3)
        s = E4M3[si].astype(np.float32)
        d = s * st
        codes = nearest(np.where(s > 0, np.abs(b) / np.where(s > 0, d, np.float32(1)), 0), E2M1)
        v = np.copysign(E2M1[codes] * s.astype(np.float64), np.where(s > 0, b, 0)) * np.float64(st)
    v = np.where(np.isfinite(amax), v, np.nan)
    return v.reshape(x.shape)


def turns(positions, freqs):
    """Angles in radians, [tokens][pairs]: pos * f modulo one turn in exact integers."""
    out = np.zeros((len(positions), len(freqs)))
    for t, p in enumerate(positions):
        for i, f in enumerate(freqs):
            out[t, i] = ((int(p) * (int(f) % 2 ** 64)) % 2 ** 64) / 2.0 ** 64
    return out * 2 * math.pi


def rope(x, positions, freqs, interleaved, magnitude=1.0, inverse=False):
    """x float64 [tokens][heads][d]: (turned, the magnitudes |a| + |b| that its error scales with)."""
    rot = 2 * len(freqs)
    angle = turns(positions, freqs)[:, None, :] * (-1 if inverse else 1)
    c, s = np.cos(angle) * magnitude, np.sin(angle) * magnitude
    first = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    second = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    y, size = np.array(x, np.float64), np.abs(np.array(x, np.float64))
    a, b = y[..., first].copy(), y[..., second].copy()
    y[..., first], y[..., second] = a * c - b * s, a * s + b * c
    both = (np.abs(a) + np.abs(b)) * abs(magnitude)
    size[..., first], size[..., second] = both, both
    return y, size


# fp32 sine and cosine (2.5 half steps), times the magnitude, two products and a sum: at most five half steps of
# magnitude (|a| + |b|).  The table's and the phase's own errors (2^-33 turns) are far below one.
ROPE_STEPS = 5 * U24


def attend(q, k, v, scale):
    """One row: q [g][d], k and v [n][d] float64 -> (o [g][d], lse [g], sum p|v| [g][d], scale sum|q k| [g])."""
    if k.shape[0] == 0:
        return np.zeros_like(q), np.full(q.shape[0], -np.inf), np.zeros_like(q), np.zeros(q.shape[0])
    s = q @ k.T * scale
    m = s.max(-1, keepdims=True)
    p = np.exp(s - m)
    total = p.sum(-1, keepdims=True)
    size = (np.abs(q) @ np.abs(k).T * scale).max(-1)
    return p @ v / total, (m + np.log(total))[:, 0], p @ np.abs(v) / total, size


def attend_bounds(size, n, d, o, pv, lse, fmt, v=None):
    """How far a bf16 output and an fp32 lse may be off.

    Scores: d exact products summed in fp32, then a product and a sum: (d + 4) half steps of sum |q k|.  A term
    exp(s - m) is off by that, by four half steps of the exponential, and by its rounding for the matrix cores (two bf16
    parts, 2^-17; for format 2 one f16 number, 2^-12); sums over n tokens by n half steps.  A quotient of two such sums is off by twice as much of sum p |v|; then one rounding to bf16.
    An f16 number's last step is 2^-24, and the row's largest term is held at 2^11 or more: smaller terms are off by half
    a step, 2^-36 of the largest, however small they are.  The sum of terms is at least the largest, so that with the
    values given ([n][d]) this comes to 2^-36 sum |v| at most."""
    ds = (d + 4) * U24 * size
    term = ds + 4 * U24 + (2.0 ** -12 if fmt == 2 else 2.0 ** -17) + (n + 8) * U24
    small = 2.0 ** -36 * np.abs(v).sum(0) if fmt == 2 and v is not None else 0.0
    return 2.0 ** -8 * np.abs(o) + 2 * term[:, None] * pv + small + 1e-30, ds + (n + 8) * U24 + 4 * U24 * (1 + np.abs(np.where(np.isfinite(lse), lse, 0)))
