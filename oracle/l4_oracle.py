"""Float64 definitions of the 4-bit latent cache, the attention mass and the
eviction (the contract of include/dsa_l4.h), written from the formulas with
NumPy.  Test infrastructure only: the library never calls it.

Row format: L[c] = 2^e * s[c // 16] * v[c]; bytes: W / 2 codes (even column in
the low nibble), W / 16 E4M3 scales, e + 127, zeros up to a multiple of 16.
"""

from __future__ import annotations

import numpy as np

from oracle.dsa_oracle import e4m3_to_f64

BLOCK = 16
MAX_EXP = 60
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = e4m3_to_f64(np.arange(0x7F, dtype=np.uint8))  # the finite values >= 0, ascending


def row_bytes(W: int) -> int:
    return -(-(W // 2 + W // BLOCK + 1) // 16) * 16


def _nearest(a: np.ndarray, grid: np.ndarray) -> np.ndarray:
    """Index of the grid value nearest to a >= 0; halfway goes to the even index
    (the codes of both formats end in the last mantissa bit), saturating."""
    a = np.minimum(a, grid[-1])
    hi = np.searchsorted(grid, a)
    lo = np.maximum(hi - 1, 0)
    up, down = grid[hi] - a, a - grid[lo]
    return np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))


def row_exponent(amax: np.ndarray) -> np.ndarray:
    """Least e in [-60, 60] with amax <= 2688 * 2^e (60 where none is); 0 for amax = 0."""
    bounds = 2688.0 * 2.0 ** np.arange(-MAX_EXP, MAX_EXP)
    e = -MAX_EXP + (np.asarray(amax, np.float64)[..., None] > bounds).sum(-1)
    return np.where(np.asarray(amax) == 0, 0, e)


def quantise(x: np.ndarray):
    """Rows x [n, W] -> (packed rows [n, row_bytes] uint8, their values [n, W] float64)."""
    x = np.asarray(x, np.float64)
    n, W = x.shape
    e = row_exponent(np.abs(x).max(1))
    y = np.ldexp(x, -e[:, None]).reshape(n, W // BLOCK, BLOCK)
    si = _nearest(np.abs(y).max(2) / 6.0, E4M3)
    s = E4M3[si][:, :, None]
    live = s > 0
    code = np.where(live, _nearest(np.abs(y) / np.where(live, s, 1.0), E2M1), 0)
    code = code + 8 * ((y < 0) & live)
    code = code.reshape(n, W).astype(np.uint8)
    out = np.zeros((n, row_bytes(W)), np.uint8)
    out[:, :W // 2] = code[:, 0::2] | (code[:, 1::2] << 4)
    out[:, W // 2:W // 2 + W // BLOCK] = si.astype(np.uint8)
    out[:, W // 2 + W // BLOCK] = e + 127
    return out, dequantise(out, W)


def dequantise(rows: np.ndarray, W: int) -> np.ndarray:
    """Packed rows [..., row_bytes] -> float64 values [..., W]."""
    rows = np.asarray(rows, np.uint8)
    code = np.empty(rows.shape[:-1] + (W,), np.uint8)
    code[..., 0::2] = rows[..., :W // 2] & 15
    code[..., 1::2] = rows[..., :W // 2] >> 4
    v = E2M1[code & 7] * np.where(code >= 8, -1.0, 1.0)
    s = e4m3_to_f64(rows[..., W // 2:W // 2 + W // BLOCK])
    e = np.clip(rows[..., W // 2 + W // BLOCK].astype(np.int64) - 127, -MAX_EXP, MAX_EXP)
    return np.ldexp(v * np.repeat(s, BLOCK, axis=-1), e[..., None])


def attention(q: np.ndarray, L: np.ndarray, R: int, scale: float):
    """(out [H, R], lse [H], p [H, m]) of one row's queries q [H, W] over rows L [m, W]."""
    if len(L) == 0:
        return np.zeros((len(q), R)), np.full(len(q), -np.inf), np.zeros((len(q), 0))
    z = scale * (q @ L.T)
    m = z.max(1, keepdims=True)
    w = np.exp(z - m)
    l = w.sum(1, keepdims=True)
    return (w / l) @ L[:, :R], (m + np.log(l))[:, 0], w / l


def add_mass(mass: np.ndarray, pos: np.ndarray, q, L, lse, scale: float) -> None:
    """Add one row's head-summed weights exp(z - lse) at its kept positions (a
    position held twice counts twice; a head with lse = -inf adds nothing)."""
    z = scale * (np.asarray(q, np.float64) @ L.T)
    live = np.isfinite(lse)
    w = np.exp(z[live] - np.asarray(lse, np.float64)[live][:, None]).sum(0)
    np.add.at(mass, pos, w)


def evict_keep(mass: np.ndarray, budget: int, sinks: int, recent: int) -> np.ndarray:
    """The positions that a sequence with these masses keeps, ascending."""
    n = len(mass)
    rank = np.where(np.isnan(mass), -np.inf, np.minimum(mass, np.finfo(np.float32).max))
    rank = rank.astype(np.float64)
    rank[:sinks] = np.inf
    rank[max(0, n - recent):] = np.inf
    return np.sort(np.argsort(-rank, kind="stable")[:min(budget, n)])
