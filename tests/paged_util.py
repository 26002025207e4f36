"""Plain 64-bit forms of the paged 4-bit cache, for its tests (no code shared
with the library): the format as include/tq.h states it, and attention by its
definition, a query at a time."""
import math

import numpy as np
import torch

SCALES = np.array([b * 2.0 ** -17 if b < 8 else (8 + b % 8) * 2.0 ** (b // 8 - 18) for b in range(224)])


def quantise(x):
    """x [..., d] (any float tensor) -> codes in -8..7 and scale bytes, numpy."""
    x = x.detach().cpu().double().numpy()
    x = np.where(np.isfinite(x).all(-1, keepdims=True), x, 0.0)
    g = x.reshape(*x.shape[:-1], -1, 32)
    byte = np.minimum(np.searchsorted(7.5 * SCALES, np.abs(g).max(-1)), 223)
    s = SCALES[byte][..., None]
    c = np.sign(g) * np.floor(np.abs(g) / np.where(s > 0, s, 1.0) + 0.5)
    return np.clip(c, -8, 7).astype(np.int64).reshape(x.shape), byte.astype(np.uint8)


def values(c, byte):
    return (c.reshape(*c.shape[:-1], -1, 32) * SCALES[byte][..., None]).reshape(c.shape)


def pack_page_rows(c, byte):
    """codes [..., d], bytes [..., d/32] -> packed code bytes [..., d/2], scale bytes."""
    u = (c + 8).astype(np.uint8)
    return u[..., 0::2] | (u[..., 1::2] << 4), byte


def page_row(pool, page_size, d, slot):
    """pool uint8 [n_pages, H, page_bytes] (numpy), one slot -> (code bytes [H, d/2], scale bytes [H, d/32])."""
    p, t = divmod(int(slot), page_size)
    rows = pool[p]
    return rows[:, t * d // 2:(t + 1) * d // 2], rows[:, page_size * d // 2 + t * d // 32: page_size * d // 2 + (t + 1) * d // 32]


def row_values(pool, page_size, d, slots):
    """Values at slots [n] -> float64 [n, H, d]."""
    p, t = np.asarray(slots) // page_size, np.asarray(slots) % page_size
    n, H, _ = pool.shape
    codes = pool[..., :page_size * d // 2].reshape(n, H, page_size, d // 2)[p, :, t]
    byte = pool[..., page_size * d // 2:].reshape(n, H, page_size, d // 32)[p, :, t]
    c = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], d).astype(np.int64) - 8
    return values(c, byte)


def attention(kpool, vpool, page_size, q, table, lens, starts, window=0, sinks=0, scale=None):
    """q [total, Hq, d] (tensor); table, lens, starts: numpy.  -> float64 [total, Hq, d], nan in rows of no sequence."""
    total, hq, d = q.shape
    qs = q.detach().cpu().double().numpy()
    out = np.full(qs.shape, np.nan)
    scale = scale or 1.0 / math.sqrt(d)
    for b in range(len(lens)):
        n, a, e = int(lens[b]), int(starts[b]), int(starts[b + 1])
        t = np.arange(n)
        if n:
            slots = table[b, t // page_size].astype(np.int64) * page_size + t % page_size
            k, v = (row_values(x, page_size, d, slots) for x in (kpool, vpool))
        for i in range(a, e):
            p = n - (e - a) + (i - a)
            see = t <= p
            if window:
                see &= (t > p - window) | (t < sinks)
            if not see.any():
                out[i] = 0.0
                continue
            for h in range(hq):
                j = h // (hq // k.shape[1])
                s = k[see, j] @ qs[i, h] * scale
                w = np.exp(s - s.max())
                out[i, h] = w @ v[see, j] / w.sum()
    return out


def bound(ref, dtype, vmax):
    """How far an output may be from `ref`: its own rounding (half a step) and
    the weights' (half a step of binary16, 2^-11 relative each, so at most
    2^-11 of the largest |v|; and weights below 2^-20 of the largest are off
    by up to 2^-31 of it, at most 2^-11 again over 2^20 tokens), plus 2^-14
    of it for the float32 scores and exponentials."""
    return np.abs(ref) * (torch.finfo(dtype).eps / 2) + vmax * (2 * 2.0 ** -11 + 2.0 ** -14) + 2.0 ** -25
