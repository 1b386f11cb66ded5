"""Plain references (numpy, 64 bits, no GPU) for the calls that say which rows of a
cache count, and batches to run them on."""
from __future__ import annotations

import numpy as np

from rows_reference import bf16_bits, bf16_value


def visible(n, Q, j, window, sinks):
    """Rows that query token j of a sequence of n rows attends to."""
    last = n - Q + j
    i = np.arange(last + 1)
    return i if not window else i[(i < sinks) | (i > last - window)]


def attention(q, k, v, scale, group, window=0, sinks=0, rounded_weights=False):
    """One sequence in 64 bits. q: [Q][Hq][D]; k, v: [n][Hkv][D]. Returns the output,
    each row's weight summed over tokens and heads ([n][Hkv]), and bounds of what fp32
    arithmetic may be off by, rounding of the output not counted:
      d    a score's absolute error: D products summed in fp32, D 2^-23 |scale| sum |q k|,
           and 2^-16 for the exponentials and rescalings of up to 64 steps; each weight
           is off by 2 d of itself (its own and the sum's)
      out  2 d sum w |v|, 2^-14 sum w |v| for sums of up to 2^10 terms, and with
           rounded_weights (bf16 tensor-core products) 2^-8 sum w |v|
      row  (2 d + 2^-14) w
    """
    Q, hq, D = q.shape
    n, hkv = k.shape[:2]
    out, weight = np.zeros((Q, hq, D)), np.zeros((n, hkv))
    out_tol, weight_tol = np.zeros((Q, hq, D)), np.zeros((n, hkv))
    if n == 0:
        return out, weight, out_tol, weight_tol
    for j in range(Q):
        see = visible(n, Q, j, window, sinks)
        for qh in range(hq):
            h = qh // group
            x, kk, vv = q[j, qh], k[see, h], v[see, h]
            s = scale * (kk @ x)
            w = np.exp(s - s.max())
            w /= w.sum()
            size = abs(scale) * (np.abs(kk) @ np.abs(x))
            d = D * 2.0 ** -23 * size.max() + 2.0 ** -16
            out[j, qh] = w @ vv
            out_tol[j, qh] = (2 * d + 2.0 ** -14 + (2.0 ** -8 if rounded_weights else 0)) * (w @ np.abs(vv))
            weight[see, h] += w
            weight_tol[see, h] += (2 * d + 2.0 ** -14) * w
    return out, weight, out_tol, weight_tol


def kept_rows(weights, n, keep, sinks, recent):
    """Indices of the rows that stay of one sequence and KV head, in order."""
    keep = min(keep, n)
    first, last = min(n, sinks), max(min(n, sinks), n - recent)
    more = keep - first - (n - last)
    w = np.where(np.isnan(weights[first:last]), -np.inf, weights[first:last]) + 0.0
    order = sorted(range(last - first), key=lambda i: (-w[i], i))[:more]
    return list(range(first)) + sorted(first + i for i in order) + list(range(last, n))


def verify(target, draft, tokens, uniforms, count):
    """(accepted, drawn token) of one sequence, and how near the nearest decision is:
    the smallest distance of a uniform number from a border, in units of it."""
    V = target.shape[1]
    near = 1.0
    for i in range(count):
        x = tokens[i]
        q = np.eye(1, V, x)[0] if draft is None else draft[i].astype(np.float64)
        p = target[i].astype(np.float64)
        near = min(near, abs(uniforms[i] * q[x] - p[x]) / max(q[x], 1e-30))
        if not uniforms[i] * q[x] < p[x]:
            r = np.where(p > q, p - q, 0.0)
            r = r if r.sum() > 0 else np.where(p > 0, p, 0.0)
            break
    else:
        i, r = count, np.where(target[count] > 0, target[count], 0.0).astype(np.float64)
    run = np.cumsum(r)
    border = uniforms[-1] * run[-1]
    near = min(near, np.abs(run / run[-1] - uniforms[-1]).min())
    return i, int(np.argmax(run > border)), near


class Cache:
    """Sequences in a paged pool: random block order, rows that belong to nobody NaN
    (as bits), and the values in 64 bits."""

    def __init__(self, lens, hkv, D, dtype="bf16", bs=16, seed=0, spare=3, width=None):
        r = np.random.default_rng(seed)
        self.lens, self.hkv, self.D, self.dtype, self.bs = list(lens), hkv, D, dtype, bs
        blocks = [-(-n // bs) for n in lens]
        self.num_blocks = sum(blocks) + spare
        self.width = width or max(1, max(blocks))
        free = r.permutation(self.num_blocks)
        self.table = np.full((len(lens), self.width), -1, np.int32)
        at = 0
        for s, b in enumerate(blocks):
            self.table[s, :b] = free[at:at + b]
            at += b
        self.free = free[at:]
        self.k = [self._values(r, (n, hkv, D)) for n in lens]
        self.v = [self._values(r, (n, hkv, D)) for n in lens]
        self.random = r

    def _values(self, r, shape):
        x = r.standard_normal(shape).astype(np.float32)
        return bf16_value(bf16_bits(x)).astype(np.float64) if self.dtype == "bf16" else x.astype(np.float64)

    def queries(self, Q, hq, gain=1.0):
        return gain * self._values(self.random, (len(self.lens), Q, hq, self.D))

    def place(self, rows, fill=np.nan):
        """[NB][Hkv][bs][D] fp32 pool of per-sequence rows."""
        pool = np.full((self.num_blocks, self.hkv, self.bs, self.D), fill, np.float32)
        for s, x in enumerate(rows):
            i = np.arange(len(x))
            pool[self.table[s, i // self.bs], :, i % self.bs] = x
        return pool

    def upload(self, values):
        import torch
        t = torch.from_numpy(np.ascontiguousarray(values, dtype=np.float32)).cuda()
        return t.bfloat16() if self.dtype == "bf16" else t


def slot_rows(pool, table, n, bs):
    """Rows 0 .. n - 1 of a sequence out of a pool [NB][Hkv][bs][...]: [n][Hkv][...]."""
    i = np.arange(n)
    return pool[np.asarray(table)[i // bs], :, i % bs]
