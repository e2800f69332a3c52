"""Definitions of the RMS norm and of the 4-bit g128 linear layer in NumPy
float64, as plain and slow as they read.  Shares no code with the CUDA path.

4-bit codes: c = q + 8, q in -8..7; byte i of a row holds k = 2i in its low
nibble and k = 2i + 1 in its high one; one fp16 scale per 128 weights."""
from __future__ import annotations

import numpy as np

from oracle import ternary_oracle as orc


def rms_norm(h, weight, eps, signs=None):
    """n_k = h_k w_k / sqrt(mean h^2 + eps) of the rows of h, rotated when signs are given."""
    h = np.asarray(h, dtype=np.float64)
    n = h / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps)
    if weight is not None:
        n = n * np.asarray(weight, dtype=np.float64)
    return orc.rotate(n, signs) if signs is not None else n


def group_scales(n, group, top):
    """max|n| / top of every run of `group` values: [M, K / group]."""
    m, k = n.shape
    return np.abs(n).reshape(m, k // group, group).max(axis=2) / top


def pack(codes):
    c = np.asarray(codes, dtype=np.int64) + 8
    assert c.min() >= 0 and c.max() <= 15
    return (c[:, 0::2] + 16 * c[:, 1::2]).astype(np.uint8)


def unpack(packed, n, k):
    b = np.asarray(packed, dtype=np.int64).reshape(n, k // 2)
    q = np.empty((n, k), dtype=np.int64)
    q[:, 0::2] = b % 16 - 8
    q[:, 1::2] = b // 16 - 8
    return q.astype(np.int8)


def prepare_weights(w, signs=None):
    """(codes, fp16 scales) of a dense matrix; signs: fold the rotation first."""
    w = np.asarray(w, dtype=np.float64)
    if signs is not None:
        w = orc.fold_weights(w, signs)
    n, k = w.shape
    g = w.reshape(n, k // 128, 128)
    top = (np.abs(g).max(axis=2) / 7.0).astype(np.float32)
    s = np.minimum(top, np.float32(8188.0)).astype(np.float16)
    d = s.astype(np.float64)[:, :, None]
    q = np.where(d > 0, np.clip(np.rint(g / np.where(d > 0, d, 1.0)), -8, 7), 0)
    return q.reshape(n, k).astype(np.int8), s


def dequantize(codes, scales):
    return codes.astype(np.float64) * np.repeat(np.asarray(scales, dtype=np.float64), 128, axis=1)


def linear(x, codes, scales, x_scales=None, signs=None):
    """x' W^T; x_scales [M, K / group] of an 8-bit x."""
    x = np.asarray(x, dtype=np.float64)
    if x_scales is not None:
        s = np.asarray(x_scales, dtype=np.float64)
        x = x * np.repeat(s, x.shape[1] // s.shape[1], axis=1)
    if signs is not None:
        x = orc.rotate(x, signs)
    return x @ dequantize(codes, scales).T
