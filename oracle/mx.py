"""Microscaled (MX) operands, the norm with the residual's addition and the rows in expert order,
in float64 (test infrastructure; see oracle/__init__). Plain definitions:

* an MX row is K elements (e2m1 nibbles or e4m3 bytes) with one UE8M0 byte per 32 of them; value =
  element * 2**(b - 127); byte 255 and the e4m3 NaNs are NaN.
* quantisation: b is the least byte in 0..254 with max|x| <= m * 2**(b - 127), m = 6 or 448; an
  element is the nearest grid value to x / 2**(b - 127), of two equally near ones that with the
  even code; the sign bit is x's. Blocks with an infinity or a NaN: b = 255, codes 0.
* norm: h = x + r, n = h / sqrt(mean h^2 + eps) * gamma.
* rows: pair p = t * top_k + j; the rows are the pairs stably sorted by expert, pairs of no expert
  last; pos[t, j] is the row of the pair, or -1 - row.
Pinned by tests/test_oracle_mx.py.
"""
import numpy as np

from .formats import E2M1_MAGNITUDE, unpack_e2m1
from .forward import _e4m3_table

E2M1, E4M3 = 0, 1
_MAGNITUDES = {E2M1: np.array(E2M1_MAGNITUDE, dtype=np.float64), E4M3: _e4m3_table()[:127].astype(np.float64)}


def value(codes, scales, fmt):
    """codes, scales (uint8 arrays of rows) -> float64 values [R, K]."""
    if fmt == E2M1:
        c = unpack_e2m1(codes)
        v = np.where(c & 8, -1.0, 1.0) * _MAGNITUDES[E2M1][c & 7]
    else:
        c = np.asarray(codes)
        mag = np.append(_MAGNITUDES[E4M3], np.nan)
        v = np.where(c & 128, -1.0, 1.0) * mag[c & 127]
    s = np.asarray(scales).astype(np.int64)
    return v * np.repeat(np.where(s == 255, np.nan, np.ldexp(1.0, s - 127)), 32, axis=-1)


def quantize(x, fmt):
    """float64 [R, K] -> (codes, scales) uint8."""
    x = np.asarray(x, dtype=np.float64)
    R, K = x.shape
    mags = _MAGNITUDES[fmt]
    limits = mags[-1] * np.ldexp(1.0, np.arange(255) - 127)
    mid = (mags[1:] + mags[:-1]) / 2
    blocks = x.reshape(R, K // 32, 32)
    finite = np.isfinite(blocks).all(-1)
    v = np.where(finite[..., None], blocks, 0.0)
    b = np.searchsorted(limits, np.abs(v).max(-1))               # least index with limit >= max
    t = np.abs(v) / np.ldexp(1.0, b - 127)[..., None]
    lo = np.searchsorted(mid, t, side="left")                    # midpoints below t
    tie = (lo < len(mid)) & (t == mid[np.minimum(lo, len(mid) - 1)])
    code = lo + (tie & (lo % 2 == 1)) + np.signbit(v) * (8 if fmt == E2M1 else 128)   # of a tie the even one
    codes = np.where(finite[..., None], code, 0).astype(np.uint8).reshape(R, K)
    scales = np.where(finite, b, 255).astype(np.uint8)
    if fmt == E2M1:
        return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8), scales
    return codes, scales


def norm(x, residual, gamma, eps):
    """(h, n) in float64."""
    h = np.asarray(x, np.float64) if residual is None else np.asarray(x, np.float64) + np.asarray(residual, np.float64)
    return h, h / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps) * np.asarray(gamma, np.float64)


def order(ids, E):
    """(offsets [E + 1], perm [P], pos [T, top_k]) of topk_ids [T, top_k]."""
    flat = np.asarray(ids).reshape(-1).astype(np.int64)
    key = np.where((flat >= 0) & (flat < E), flat, E)
    perm = np.argsort(key, kind="stable")
    pos = np.empty(len(flat), np.int64)
    pos[perm] = np.arange(len(flat))
    offsets = np.array([(key < e).sum() for e in range(E + 1)])
    pos = np.where(key < E, pos, -1 - pos)
    return offsets.astype(np.int32), perm.astype(np.int32), pos.reshape(np.shape(ids)).astype(np.int32)


def unpermute(rows, pos, w):
    """sum_j w[t, j] rows[pos[t, j]] and the sum of the terms' magnitudes, float64."""
    rows = np.asarray(rows, np.float64)
    here = pos >= 0
    v = rows[np.where(here, pos, 0)] * np.where(here, 1.0 if w is None else np.where(here, w, 0.0), 0.0)[..., None]
    v = np.where(here[..., None], v, 0.0)
    return v.sum(1), np.abs(v).sum(1)
