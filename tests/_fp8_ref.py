"""Plain 64-bit reference of the 8-bit paged cache (include/bdfp8.h), written from
the header: code values, page layouts, the append and the attention."""
from __future__ import annotations

import numpy as np
import torch

from fp4_kv_cache_quant_b200 import bdfp8

PAGE, BLOCK = 64, 16
TOP = {bdfp8.E4M3: 448.0, bdfp8.E5M2: 57344.0}


def code_values(fmt: int) -> np.ndarray:
    """The 256 values of E4M3 (no infinity, code 127 a NaN) or E5M2."""
    ebits, mbits, bias = (4, 3, 7) if fmt == bdfp8.E4M3 else (5, 2, 15)
    v = np.zeros(256)
    for c in range(256):
        e, m = (c >> mbits) & ((1 << ebits) - 1), c & ((1 << mbits) - 1)
        x = m * 2.0 ** (1 - bias - mbits) if e == 0 else (1 + m / 2 ** mbits) * 2.0 ** (e - bias)
        if fmt == bdfp8.E4M3 and c & 127 == 127:
            x = np.nan
        elif fmt == bdfp8.E5M2 and e == 31:
            x = np.nan if m else np.inf
        v[c] = -x if c & 128 else x
    return v


def k_offset(slot, elem, d):
    return slot // 8 * 8 * d + elem // 16 * 128 + slot % 8 * 16 + elem % 16


def v_offset(slot, chan):
    return chan // 8 * 512 + slot // 16 * 128 + chan % 8 * 16 + slot % 16


def offsets(d):
    s, e = np.arange(PAGE)[:, None], np.arange(d)[None, :]
    return k_offset(s, e, d), v_offset(s, e)


def codes_of(cache) -> tuple[np.ndarray, np.ndarray]:
    """(keys, values) codes [num_pages, H_kv, 64, d]."""
    ko, vo = offsets(cache.d)
    return cache.k_pages.cpu().numpy()[:, :, ko], cache.v_pages.cpu().numpy()[:, :, vo]


def values_of(cache) -> tuple[np.ndarray, np.ndarray]:
    """(keys, values) as the 64-bit numbers they stand for [num_pages, H_kv, 64, d]."""
    t = code_values(cache.fmt)
    sc = cache.kv_scales.cpu().numpy().astype(np.float64)
    out = []
    for which, c in enumerate(codes_of(cache)):
        with np.errstate(invalid="ignore"):
            out.append(t[c] * np.repeat(sc[:, :, which], BLOCK, axis=2)[..., None])
    return tuple(out)


def attention(q, K, V, block_table, seq_lens, sm_scale, window=0, sinks=0):
    """-> (out, tol) [B, T_q, H_q, d] fp64.  q as fp64; K, V from values_of.  Pages outside the
    cache and tokens a row does not see are left out.

    tol is what the kernel may be off by: half a bf16 step of the result (2^-8 |out|) and, with A =
    sum_t p_t |v_t| and D = sm_scale max_t sum_i |q_i k_ti|, A times
      2^-9 + 2^-11       a probability's three E5M2 terms (half steps of 2^-3 each) and its fp16 form
      2 (d + 8) 2^-23 D  the logits' fp32 sums (a whole step per addition), in p and in the sum of p
      (n + 64) 2^-23     the fp32 sums over n tokens
      2^-20              the exponential (2 units of 2^-22 twice) and the final product
    and n 2^-28 max|v|: the terms' floor, 2^-28 of the largest scaled probability, times a code.
    The query's terms leave 2^-17 of a row's largest element at the most: with that as an error of every
    q_i, 2 * 2^-17 max|q| sm_scale max_t sum_i |k_ti| in p and in the sum of p."""
    B, T, Hq, d = q.shape
    H = K.shape[1]
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(B):
        N = int(seq_lens[b])
        if N <= 0 or N > block_table.shape[1] * PAGE:
            continue
        pages = block_table[b, np.arange(N) // PAGE]
        good = (pages >= 0) & (pages < K.shape[0])
        slots = np.arange(N) % PAGE
        pg = np.where(good, pages, 0)
        for i in range(T):
            p = N - T + i
            t = np.arange(N)
            see = good & (t <= p)
            if window > 0:
                see &= (t > p - window) | (t < sinks)
            if not see.any():
                continue
            for h in range(Hq):
                k = K[pg[see], h * H // Hq, slots[see]]
                v = V[pg[see], h * H // Hq, slots[see]]
                x = k @ q[b, i, h] * sm_scale
                e = np.exp(x - x.max())
                e /= e.sum()
                out[b, i, h] = e @ v
                A = e @ np.abs(v)
                D = abs(sm_scale) * (np.abs(k) @ np.abs(q[b, i, h])).max()
                D += 2.0 ** 23 / (d + 8) * 2.0 ** -17 * np.abs(q[b, i, h]).max() * abs(sm_scale) * np.abs(k).sum(1).max()
                n = see.sum()
                rel = 2.0 ** -9 + 2.0 ** -11 + 2 * (d + 8) * 2.0 ** -23 * D + (n + 64) * 2.0 ** -23 + 2.0 ** -20
                tol[b, i, h] = 2.0 ** -8 * np.abs(out[b, i, h]) + A * rel + n * 2.0 ** -28 * np.abs(v).max()
    return out, tol


def scale_of(amax: np.ndarray, fmt: int) -> np.ndarray:
    """The smallest power of two s >= 2^-126 with amax <= top s; 1 for 0."""
    with np.errstate(divide="ignore"):
        e = np.where(amax > 0, np.ceil(np.log2(np.where(amax > 0, amax, 1) / TOP[fmt])), 0)
    s = 2.0 ** e
    s = np.where((amax > 0) & (amax <= TOP[fmt] * s / 2), s / 2, s)
    s = np.where(amax > TOP[fmt] * s, s * 2, s)
    return np.where(amax > 0, np.maximum(s, 2.0 ** -126), 1.0)


def rotate(x, cos_sin_rows, interleaved):
    """x [n, H, d] fp64 rotated by rows [n, rot] of (cosines, sines), in 64 bits."""
    rot = cos_sin_rows.shape[1]
    y = x.copy()
    c, s = cos_sin_rows[:, None, : rot // 2], cos_sin_rows[:, None, rot // 2:]
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


class AppendRef:
    """What the cache holds after appends: per sequence every token's rotated key and value, in
    fp32 (one rounding of the 64-bit rotation), quantized block by block."""

    def __init__(self, B, H, d, fmt):
        self.B, self.H, self.d, self.fmt = B, H, d, fmt
        self.k = [np.zeros((0, H, d), np.float32) for _ in range(B)]
        self.v = [np.zeros((0, H, d), np.float32) for _ in range(B)]

    def append(self, b, k, v, cos_sin=None, positions=None, interleaved=False):
        n0 = len(self.k[b])
        pos = np.arange(n0, n0 + len(k)) if positions is None else positions
        k = k.astype(np.float64)
        if cos_sin is not None:
            k = rotate(k, cos_sin[pos].astype(np.float64), interleaved)
        self.k[b] = np.concatenate([self.k[b], k.astype(np.float32)])
        self.v[b] = np.concatenate([self.v[b], v.astype(np.float32)])

    def blocks(self, b):
        """[(index of block, codes and scales of keys, of values)] as (codes [H, 16, d], scale [H])."""
        got = []
        f8 = bdfp8.DTYPES[self.fmt]
        for i in range(0, len(self.k[b]), BLOCK):
            pair = []
            for x in (self.k[b], self.v[b]):
                blk = np.zeros((BLOCK, self.H, self.d), np.float32)
                part = x[i: i + BLOCK]
                blk[: len(part)] = part
                s = scale_of(np.abs(blk).max((0, 2)).astype(np.float64), self.fmt)
                c = torch.from_numpy((blk / s[None, :, None]).astype(np.float32)).to(f8).view(torch.uint8).numpy()
                pair.append((c.transpose(1, 0, 2), s))
            got.append((i // BLOCK, *pair))
        return got
