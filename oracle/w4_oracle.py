"""CPU oracle of the 4-bit group-scale linear (numpy, 64 bits).

W[n,k] = S[n, k // group] * c[n,k], c in -8 .. 7, the last group of a row may
be short; y[m,n] = sum over groups of S * (sum of c * x). Quantisation: per
group a = max|w|, S = RN32(a / 7) (rounded once more to bf16 for bf16 scales),
c = clamp(rint(RN32(w / S)), -8, 7), zeros where S is zero.
"""
from __future__ import annotations

import numpy as np

__all__ = ["w4_quantise", "w4_forward", "w4_sum_abs", "w4_nibbles", "bf16_rn"]


def bf16_rn(v: np.ndarray) -> np.ndarray:
    """fp32 -> nearest bf16 (half to even), as fp32."""
    b = np.ascontiguousarray(v, np.float32).view(np.uint32).astype(np.uint64)
    b = ((b + 0x7FFF + ((b >> 16) & 1)) >> 16) << 16
    return b.astype(np.uint32).view(np.float32)


def w4_quantise(W: np.ndarray, group: int, bf16_scales: bool = False):
    """fp32 W [N, K] -> (codes int8 [N, K], S fp32 [N, ceil(K/group)])."""
    W = np.asarray(W, np.float32)
    N, K = W.shape
    G = -(-K // group)
    codes = np.zeros((N, K), np.int8)
    S = np.zeros((N, G), np.float32)
    for g in range(G):
        w = W[:, g * group:(g + 1) * group]
        s = (np.abs(w).max(axis=1) / np.float32(7)).astype(np.float32)
        if bf16_scales:
            s = bf16_rn(s)
        S[:, g] = s
        for n in np.flatnonzero(s > 0):
            codes[n, g * group:(g + 1) * group] = np.clip(np.rint(w[n] / s[n]), -8, 7)
    return codes, S


def w4_nibbles(codes: np.ndarray) -> np.ndarray:
    """Codes [N, K] -> bytes [N, K/2], column 2j in the low nibble, stored as c + 8."""
    c = (codes.astype(np.int16) + 8).astype(np.uint8)
    return np.ascontiguousarray(c[:, 0::2] | (c[:, 1::2] << 4))


def _dequant(codes, S, group):
    K = codes.shape[1]
    return codes.astype(np.float64) * np.repeat(S.astype(np.float64), group, axis=1)[:, :K]


def w4_forward(x: np.ndarray, codes: np.ndarray, S: np.ndarray, group: int) -> np.ndarray:
    return x.astype(np.float64) @ _dequant(codes, S, group).T


def w4_sum_abs(x: np.ndarray, codes: np.ndarray, S: np.ndarray, group: int) -> np.ndarray:
    """sum |S c x| per output: what rounding errors of a sum are measured against."""
    return np.abs(x).astype(np.float64) @ np.abs(_dequant(codes, S, group)).T
