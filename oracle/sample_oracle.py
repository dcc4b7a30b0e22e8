"""CPU oracle of the sampler (numpy, integers).

Per row: tokens whose logit is NaN or -inf are out; w = exp((x - max) / T) as an
integer number of 2^-40; top-k, top-p, min-p in this order; the first kept index
whose running sum exceeds u times the kept sum.
"""
from __future__ import annotations

import math

import numpy as np

__all__ = ["sample_kept", "sample_row"]

ONE = 1 << 40


def _weights(row: np.ndarray, T: float) -> np.ndarray:
    best = row.max()
    out = np.zeros(row.size, object)
    for i, v in enumerate(row):
        if v == best:
            out[i] = ONE
        elif math.isfinite(best):
            out[i] = int(np.rint(np.exp((float(v) - float(best)) / T) * ONE)) if math.isfinite(T) else ONE
        else:
            out[i] = 0
    return out


def sample_kept(row, T=1.0, k=0, p=1.0, m=0.0):
    """(kept indexes ascending, their integer weights) of one row of fp32 values."""
    row = np.asarray(row, np.float64)
    idx = np.array([i for i, v in enumerate(row) if not math.isnan(v) and v != -math.inf], np.int64)
    if idx.size == 0:
        return idx, np.zeros(0, object)
    vals = row[idx]
    if not T > 0:
        return idx[[int(np.argmax(vals))]], np.array([ONE], object)
    idx = idx[np.argsort(-vals, kind="stable")]
    w = _weights(row[idx], float(T))
    if k > 0:
        idx, w = idx[:k], w[:k]
    if p < 1:
        need = max(float(p), 0.0) * float(int(w.sum()))
        run, n = 0, 0
        while n < idx.size and (n == 0 or run < need):
            run += int(w[n])
            n += 1
        idx, w = idx[:n], w[:n]
    if m > 0:
        keep = np.array([int(v) >= min(float(m), 1.0) * ONE for v in w])
        idx, w = idx[keep], w[keep]
    order = np.argsort(idx)
    return idx[order], w[order]


def sample_row(row, u, T=1.0, k=0, p=1.0, m=0.0):
    """(token, log-probability) of one row."""
    idx, w = sample_kept(row, T, k, p, m)
    if idx.size == 0:
        return -1, -math.inf
    total = int(w.sum())
    target = 0 if not u > 0 else (total - 1 if u >= 1 else min(int(float(u) * float(total)), total - 1))
    run = 0
    for i, v in zip(idx, w):
        run += int(v)
        if run > target:
            if not T > 0:
                return int(i), 0.0
            best = np.nanmax(np.asarray(row, np.float64))
            x = float(row[int(i)])
            d = 0.0 if x == best else (x - float(best)) / float(T)
            return int(i), d - math.log(total / ONE)
    raise AssertionError("unreachable: target < total")
