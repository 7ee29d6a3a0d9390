"""MXFP4 and the row movement's gradients in numpy float64, for the tests of
the kernels: written from the formats' definition, without the library."""
from __future__ import annotations

import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantise(v):
    """Codes (0..15) and scale bytes of blocks of 32 along the last axis."""
    v = np.asarray(v, np.float64)
    b = v.reshape(*v.shape[:-1], v.shape[-1] // 32, 32)
    a = np.abs(b).max(-1)
    finite = np.isfinite(a)
    _, ex = np.frexp(np.where(finite, a, 1.0))       # a = m * 2^ex, m in [0.5, 1)
    e = np.clip(np.where(a == 0, -127, ex - 1 - 2), -127, 127).astype(np.int64)
    m = np.abs(np.where(finite[..., None], b, 0.0)) * np.ldexp(1.0, -e)[..., None]
    dist = np.abs(m[..., None] - MAGNITUDES)
    # the nearest magnitude; of two equally near the one with the even code
    code = np.argmin(dist + 1e-12 * (np.arange(8) % 2) * (dist == dist.min(-1, keepdims=True)), -1)
    code = np.where(m >= 6.0, 7, code) + 8 * np.signbit(b)
    code = np.where(finite[..., None], code, 0)
    return code.reshape(v.shape).astype(np.uint8), np.where(finite, e + 127, 255).astype(np.uint8)


def values(codes, scales):
    """Values (float64) of codes [..., K] and scale bytes [..., K / 32]."""
    c = np.asarray(codes).astype(np.int64)
    v = MAGNITUDES[c & 7] * np.where(c & 8, -1.0, 1.0)
    s = np.asarray(scales).astype(np.int64)
    f = np.where(s == 255, np.nan, np.ldexp(1.0, s - 127))
    return (v.reshape(*v.shape[:-1], v.shape[-1] // 32, 32) * f[..., None]).reshape(v.shape)


def unpack(packed):
    p = np.asarray(packed, np.uint8)
    return np.stack((p & 15, p >> 4), -1).reshape(*p.shape[:-1], 2 * p.shape[-1])


def pack(codes):
    c = np.asarray(codes, np.uint8)
    return (c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8)


def scale_at(group, ktiles, row, block):
    """Byte of the scale of (row group, row in it, block)."""
    return (group * ktiles + block // 4) * 512 + (row % 32) * 16 + (row // 32) * 4 + block % 4


def weight_scales(buf, E, K, N):
    """Scale bytes [E, N, K / 32] out of the tiled buffer."""
    n = np.arange(N)[:, None]
    b = np.arange(K // 32)[None, :]
    buf = np.asarray(buf)
    return np.stack([buf[scale_at(e * (N // 128) + n // 128, K // 128, n % 128, b)] for e in range(E)])


def row_groups(seg):
    """(group, row in the group) of every row r < seg[-1]."""
    seg = np.asarray(seg, np.int64)
    r = np.arange(seg[-1])
    e = np.searchsorted(seg[1:], r, side="right")
    rank = r - seg[e]
    return seg[e] // 128 + e + rank // 128, rank % 128


def row_scales(buf, seg, K):
    g, r = row_groups(seg)
    return np.asarray(buf)[scale_at(g[:, None], K // 128, r[:, None], np.arange(K // 32)[None, :])]


def combine_backward(d_out, y, w, slot_to_row, rows_max):
    """dy [rows_max, d] (NaN where no slot holds the row), dw [T, k], and the
    sum of the magnitudes of each dw's terms."""
    d_out, y, w = (np.asarray(a, np.float64) for a in (d_out, y, w))
    T, k = w.shape
    s2r = np.asarray(slot_to_row).reshape(T, k)
    dy = np.full((rows_max, d_out.shape[1]), np.nan)
    dw, mag = np.zeros((T, k)), np.zeros((T, k))
    for j in range(k):
        t = np.nonzero(s2r[:, j] >= 0)[0]
        r = s2r[t, j]
        dy[r] = w[t, j][:, None] * d_out[t]
        dw[t, j] = np.sum(d_out[t] * y[r], 1)
        mag[t, j] = np.sum(np.abs(d_out[t] * y[r]), 1)
    return dy, dw, mag


def gather_backward(d_x_perm, slot_to_row, T, k, dx_in=None):
    """dx [T, d] and the sum of the magnitudes of its terms."""
    g = np.asarray(d_x_perm, np.float64)
    s2r = np.asarray(slot_to_row).reshape(T, k)
    dx = np.zeros((T, g.shape[1])) if dx_in is None else np.array(dx_in, np.float64)
    mag = np.abs(dx)
    for j in range(k):
        t = np.nonzero(s2r[:, j] >= 0)[0]
        dx[t] += g[s2r[t, j]]
        mag[t] += np.abs(g[s2r[t, j]])
    return dx, mag


def silu(g):
    return g / (1.0 + np.exp(-g))


def gelu(z):
    from scipy.special import erf
    return 0.5 * z * (1.0 + erf(z / np.sqrt(2.0)))
