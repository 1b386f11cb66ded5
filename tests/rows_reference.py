"""Plain references (numpy, no GPU) for the 4-bit cache and the norm and
rotation calls: the cache's pairs and codes in the IEEE fp32 steps that define
them, everything else in 64 bits."""
from __future__ import annotations

import numpy as np


def bf16_bits(x, mode="nearest"):
    """fp32 -> bf16 bit patterns (uint16): to nearest even, "down" or "up"."""
    b = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32)
    if mode == "nearest":
        return ((b + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint16)
    cut, rest = b >> 16, (b & 0xFFFF) != 0
    negative = (b >> 31) != 0
    away = rest & (negative if mode == "down" else ~negative)
    return (cut + away).astype(np.uint16)


def bf16_value(bits):
    return (np.asarray(bits, dtype=np.uint32) << 16).view(np.float32)


def bf16_of_double(x):
    """64-bit values rounded once to bf16 (bits)."""
    x = np.asarray(x, dtype=np.float64)
    f = x.astype(np.float32)
    # fp32 towards zero with the lost bits in the last place: rounding that to
    # bf16 is rounding x.
    over = np.abs(f.astype(np.float64)) > np.abs(x)
    f = np.where(over, np.nextafter(f, np.float32(0)), f)
    b = np.ascontiguousarray(f).view(np.uint32) | (f.astype(np.float64) != x).astype(np.uint32)
    return bf16_bits(b.view(np.float32))


def quantise4(x):
    """Codes (uint8, packed) and pairs (uint16 bf16 bits, [..., 2]) of rows x (fp32)."""
    x = np.asarray(x, dtype=np.float32)
    lo_bits = bf16_bits(x.min(-1) + np.float32(0), "down")     # a zero is +0
    lo = bf16_value(lo_bits)
    s_bits = bf16_bits((x.max(-1) - lo) / np.float32(15), "up")
    s = bf16_value(s_bits)
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.rint((x - lo[..., None]) / s[..., None])
    c = np.where(s[..., None] > 0, np.clip(c, 0, 15), 0).astype(np.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4), np.stack([lo_bits, s_bits], -1)


def codes4(packed):
    return np.stack([packed & 15, packed >> 4], -1).reshape(*packed.shape[:-1], 2 * packed.shape[-1])


def values4(packed, pairs):
    """The rows' values in 64 bits."""
    lo, s = (bf16_value(pairs[..., i]).astype(np.float64)[..., None] for i in (0, 1))
    return lo + s * codes4(packed)


def attention4(q, pools, table, n, scale, block_size, window=0):
    """One sequence's decode attention in 64 bits and the error bound of each
    output element. q: [Q][Hq][D] (64 bits); pools: k codes, v codes, k pairs,
    v pairs; n rows through `table`. The bound counts, for an output o = sum w v,
    v = lo + s c:
      2^-8 |o|                    the rounding to bf16
      2^-11 sum w s c             each weight times s rounded to f16
      2^-24 w_max sum s c         weights below f16's normal range
      2 d sum w (|lo| + s c)      a relative error d of each weight: scores are
                                  fp32 sums of about 20 terms of size
                                  |scale| (s sum |q| c + |lo| sum |q|), and the
                                  exponential adds less than that margin
    """
    Q, hq, D = q.shape
    kc, vc, kp, vp = pools
    hkv = kc.shape[1]
    G = hq // hkv
    out, tol = np.zeros((Q, hq, D)), np.zeros((Q, hq, D))
    if n == 0:
        return out, tol
    i = np.arange(n)
    blk, off = np.asarray(table)[i // block_size], i % block_size
    for h in range(hkv):
        k = values4(kc[blk, h, off], kp[blk, h, off])
        klo, ks = (bf16_value(kp[blk, h, off][:, e]).astype(np.float64) for e in (0, 1))
        kcode = codes4(kc[blk, h, off]).astype(np.float64)
        vlo, vs = (bf16_value(vp[blk, h, off][:, e]).astype(np.float64)[:, None] for e in (0, 1))
        sc = vs * codes4(vc[blk, h, off])
        for j in range(Q):
            last = n - Q + j
            first = max(0, last + 1 - window) if window else 0
            see = slice(first, last + 1)
            for g in range(G):
                x = q[j, h * G + g]
                s = scale * (k[see] @ x)
                w = np.exp(s - s.max())
                w /= w.sum()
                o = w @ (vlo[see] + sc[see])
                size = abs(scale) * (ks[see] * (kcode[see] @ np.abs(x)) + np.abs(klo[see]) * np.abs(x).sum())
                d = size.max() * 2.0 ** -18 + 2.0 ** -20
                out[j, h * G + g] = o
                tol[j, h * G + g] = (2.0 ** -8 * np.abs(o) + 2.0 ** -11 * (w @ sc[see])
                                     + 2.0 ** -24 * w.max() * sc[see].sum(0)
                                     + 2 * d * (w @ (np.abs(vlo[see]) + sc[see])))
    return out, tol


def norm_rope(x, weight, positions, cos_sin, eps=1e-6, weight_offset=0.0, interleaved=False,
              pair_axis=None):
    """Norm and rotation of x [T][H][D] in 64 bits, and |a| + |b| of the products
    that each output is the sum of (the scale of its fp32 error). positions:
    [axes][T]; cos_sin None: no rotation; weight None: no norm."""
    x = np.asarray(x, dtype=np.float64)
    y = x
    if weight is not None:
        y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (np.asarray(weight, np.float64) + weight_offset)
    out, size = y.copy(), np.abs(y)
    if cos_sin is not None:
        half = cos_sin.shape[1] // 2
        for i in range(half):
            pos = positions[pair_axis[i] if pair_axis is not None else 0]
            c, s = (cos_sin[pos, i + o].astype(np.float64)[:, None] for o in (0, half))
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            out[..., a] = y[..., a] * c - y[..., b] * s
            out[..., b] = y[..., b] * c + y[..., a] * s
            size[..., a] = np.abs(y[..., a] * c) + np.abs(y[..., b] * s)
            size[..., b] = np.abs(y[..., b] * c) + np.abs(y[..., a] * s)
    return out, size
