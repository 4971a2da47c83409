"""Float64 definitions of the key/value step: norms and rotation of query and key
heads, rows held in 4 bits, and causal attention through a sliding window with a
few first tokens that stay visible.  Plain numpy, independent of the product.
"""
from __future__ import annotations

import numpy as np


def hadamard_matrix(d: int) -> np.ndarray:
    h = np.ones((1, 1))
    while h.shape[0] < d:
        h = np.block([[h, h], [h, -h]])
    return h / np.sqrt(d)


def turn_rows(x, positions, gamma=None, norm=True, eps=1e-6, rot_dim=None, base=10000.0, hadamard=False):
    """Rows x [n, heads, d] at positions [n]: norm, rotation, Hadamard."""
    y = np.asarray(x, dtype=np.float64)
    d = y.shape[-1]
    rot_dim = d if rot_dim is None else rot_dim
    if norm:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + np.float64(np.float32(eps)))
        if gamma is not None:
            y = y * np.asarray(gamma, dtype=np.float64)
    y = y.copy()
    for i in range(rot_dim // 2):
        ang = np.asarray(positions, dtype=np.float64) * base ** (-2.0 * i / rot_dim)
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        a, b = y[..., 2 * i].copy(), y[..., 2 * i + 1].copy()
        y[..., 2 * i] = a * c - b * s
        y[..., 2 * i + 1] = a * s + b * c
    return y @ hadamard_matrix(d) if hadamard else y


def hold_rows(y):
    """(codes int8, steps fp32, t * s) of rows y [..., d] float64, with the format's fp32 steps."""
    t = np.asarray(y).astype(np.float32)
    s = np.float32(7.0) / np.maximum(np.abs(t).max(-1, keepdims=True), np.float32(1e-5))
    z = t * s
    return np.clip(np.rint(z), -8, 7).astype(np.int8), (np.float32(1.0) / s)[..., 0], z


def pack_codes(codes):
    """Codes [..., d] -> bytes [..., d/2]: code 2j + i of each 8 at bits 4j + 16i of a little-endian word."""
    u = (np.asarray(codes).astype(np.int64) & 15).reshape(*codes.shape[:-1], -1, 8)
    word = np.zeros(u.shape[:-1], dtype=np.int64)
    for j in range(4):
        for i in range(2):
            word |= u[..., 2 * j + i] << (4 * j + 16 * i)
    return word.astype("<u4").view(np.uint8).reshape(*codes.shape[:-1], -1)


def unpack_codes(packed):
    """Bytes [..., d/2] -> codes [..., d] int8."""
    word = np.ascontiguousarray(packed).view("<u4").astype(np.int64)
    out = np.empty((*word.shape, 8), dtype=np.int8)
    for j in range(4):
        for i in range(2):
            n = (word >> (4 * j + 16 * i)) & 15
            out[..., 2 * j + i] = np.where(n < 8, n, n - 16)
    return out.reshape(*packed.shape[:-1], -1)


def visible(positions, n_keys, window=0, sinks=0):
    """[queries, keys]: key j is visible at position p."""
    p = np.asarray(positions)[:, None]
    j = np.arange(n_keys)[None, :]
    see = j <= p
    if window > 0:
        see &= (j > p - window) | (j < sinks)
    return see


def attention(q, k, v, see):
    """q [n, d], k, v [T, d], see [n, T] -> (output [n, d], sum of weights times |v|,
    largest visible score error magnitude sum_i |q_i k_i| / sqrt(d) [n]); rows that
    see nothing are zero."""
    q, k, v = (np.asarray(a, dtype=np.float64) for a in (q, k, v))
    d = q.shape[-1]
    k, v = (np.where(see.any(0)[:, None], a, 0.0) for a in (k, v))
    s = np.where(see, q @ k.T / np.sqrt(d), -np.inf)
    some = see.any(-1, keepdims=True)
    w = np.where(see, np.exp(s - np.where(some, s.max(-1, keepdims=True, initial=-np.inf, where=see), 0.0)), 0.0)
    w = w / np.where(some, w.sum(-1, keepdims=True), 1.0)
    mag = np.where(see, np.abs(q) @ np.abs(k).T / np.sqrt(d), 0.0).max(-1, initial=0.0)
    return w @ v, w @ np.abs(v), mag
