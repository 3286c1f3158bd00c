"""fp64 oracle of the quantised K/V cache, of attention over it and of the
rotary positions: the definitions, element by element.

The cache's arrays are numpy uint8 codes [pages, 2, H_kv, P, D / 2] and uint16
bfloat16 bit patterns [pages, 2, H_kv, P, D / 32].
"""
from __future__ import annotations

import numpy as np

from .attention import decode

GROUP = 32


def bf16_round(x):
    """float64 -> bfloat16 bit patterns, to nearest, ties to even (finite
    values and NaN; overflow goes to infinity)."""
    x = np.asarray(x, np.float64)
    m, e = np.frexp(np.abs(x))                       # |x| = m 2^e, m in [0.5, 1)
    step = np.ldexp(1.0, np.maximum(e - 8, -133))    # 8 significant bits, subnormals from 2^-133
    r = np.rint(np.abs(x) / step) * step
    f = r.astype(np.float32)                         # exact: 8 bits
    bits = (f.view(np.uint32) >> 16).astype(np.uint16)
    bits = np.where(np.signbit(x) & (r != 0), bits | 0x8000, bits).astype(np.uint16)
    return np.where(np.isnan(x), 0x7FC0, bits).astype(np.uint16)


def quantise(x):
    """(codes n in 0..15 as [..., D] uint8, scale bits [..., D / 32]) of rows
    of finite or non-finite float64 values [..., D]."""
    g = np.asarray(x, np.float64).reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    finite = np.isfinite(g).all(-1)
    safe = np.where(np.isfinite(g), g, 0.0)
    first = np.abs(safe).argmax(-1)                  # argmax: the first of equals
    xe = np.take_along_axis(safe, first[..., None], -1)[..., 0]
    bits = bf16_round(-xe / 8)
    s = decode(bits, "bf16")
    some = finite & (s != 0)
    bits = np.where(some, bits, np.where(finite, 0, 0x7FC0)).astype(np.uint16)
    n = np.clip(np.rint(safe / np.where(some, s, 1.0)[..., None]), -8, 7) + 8
    n = np.where(some[..., None], n, 8).astype(np.uint8)
    return n.reshape(x.shape), bits


def pack(n):
    """Codes [..., D] as the cache's bytes [..., D / 2]."""
    D = n.shape[-1]
    NG = D // GROUP
    d = np.arange(D)
    word, nib = (d % GROUP) // 4 * NG + d // GROUP, d % 4
    out = np.zeros((*n.shape[:-1], D // 2), np.uint8)
    for i in range(D):
        out[..., 2 * word[i] + nib[i] // 2] |= ((n[..., i] & 15) << int(4 * (nib[i] % 2))).astype(np.uint8)
    return out


def unpack(codes):
    """The cache's bytes [..., D / 2] as codes [..., D]."""
    D = codes.shape[-1] * 2
    NG = D // GROUP
    d = np.arange(D)
    word, nib = (d % GROUP) // 4 * NG + d // GROUP, d % 4
    return (codes[..., 2 * word + nib // 2] >> (4 * (nib % 2)).astype(np.uint8)) & 15


def values(codes, scale_bits):
    """What rows of codes [..., D / 2] and scales [..., D / 32] stand for."""
    s = np.repeat(decode(scale_bits, "bf16"), GROUP, -1)
    with np.errstate(invalid="ignore"):
        return (unpack(codes).astype(np.float64) - 8) * s


def sequence_rows(codes, scale_bits, table_row, n, which):
    """Tokens 0 .. n - 1 of a sequence as float64 [n, H_kv, D]."""
    P = codes.shape[3]
    j = np.arange(n)
    pg = np.asarray(table_row)[j // P]
    return values(codes[pg, which, :, j % P], scale_bits[pg, which, :, j % P])


def attention(q, k, v, scale, window=-1):
    """One sequence: q [n, H, D] its last tokens, k, v [len, H_kv, D], all
    float64.  (O [n, H, D], LSE [H, n], and sum_j p_j |v_j| [n, H, D])."""
    n, H, D = q.shape
    L, Hkv = k.shape[:2]
    o, a = np.zeros((n, H, D)), np.zeros((n, H, D))
    lse = np.full((H, n), -np.inf)
    for i in range(n):
        pos = L - n + i
        lo = max(0, pos - window) if window >= 0 else 0
        if pos < 0:
            continue
        for h in range(H):
            kk, vv = k[lo:pos + 1, h // (H // Hkv)], v[lo:pos + 1, h // (H // Hkv)]
            z = kk @ q[i, h] * scale
            m = z.max()
            p = np.exp(z - m)
            lse[h, i] = m + np.log(p.sum())
            p /= p.sum()
            o[i, h], a[i, h] = p @ vv, p @ np.abs(vv)
    return o, lse, a


def rotary(x, positions, inv_freq, axes, interleaved=False, inverse=False):
    """x [T, H, D] float64, positions [T, A]: the turned x.  The angles are
    taken in extended precision where numpy has it."""
    F = len(inv_freq)
    ang = positions[:, axes].astype(np.longdouble) * np.asarray(inv_freq, np.longdouble)
    c, s = np.cos(ang).astype(np.float64)[:, None], np.sin(ang).astype(np.float64)[:, None]
    if inverse:
        s = -s
    f = np.arange(F)
    a, b = (2 * f, 2 * f + 1) if interleaved else (f, f + F)
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y
