"""Norm and rotation, the 8-bit block cache and its attention -- oracle (test infrastructure only), fp64.

The method descriptions have no counterpart for these; the definitions are the
textbook ones (RMS norm, rotary position embedding, softmax attention) and the
cache format that include/svsa.h states.

  norm_rope      y = R(p) (x / sqrt(mean(x^2) + eps) * w), R turning the pairs
  encode/decode  8-bit codes under power-of-two scales, nearest value, ties to
                 the even code
  BlockCache     pages of one 64-token block per head, appended token ranges
  select_blocks  exact (rational) scores from whole numbers and powers of two
  cache_attention  materialised softmax over the keys a query sees
"""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

BLOCK = 64


# ---- norm and rotation ------------------------------------------------------

def _pairs(d: int, halves: bool):
    i = np.arange(d // 2)
    return (i, i + d // 2) if halves else (2 * i, 2 * i + 1)


def norm_rope(x, w, cos, sin, halves: bool, eps: float):
    """x [..., d]; w [d]; cos, sin [..., d/2] of each row's pairs (None: no rotation)."""
    x = np.asarray(x, dtype=np.float64)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    if cos is None:
        return y
    a, b = _pairs(x.shape[-1], halves)
    out = np.empty_like(y)
    out[..., a] = y[..., a] * cos - y[..., b] * sin
    out[..., b] = y[..., a] * sin + y[..., b] * cos
    return out


def norm_rope_bwd(g, x, w, cos, sin, halves: bool, eps: float):
    """(dx, dw per row): gradients of sum(g * norm_rope(x, w)) with respect to x and to w (not summed over rows)."""
    g, x = np.asarray(g, dtype=np.float64), np.asarray(x, dtype=np.float64)
    d = x.shape[-1]
    if cos is not None:
        a, b = _pairs(d, halves)
        t = np.empty_like(g)
        t[..., a] = g[..., a] * cos + g[..., b] * sin
        t[..., b] = g[..., b] * cos - g[..., a] * sin
        g = t
    s = np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x / s
    gw = g * w
    return (gw - n * (gw * n).mean(-1, keepdims=True)) / s, g * n


# ---- 8-bit codes ------------------------------------------------------------

def e4m3_value(code: int) -> float:
    """The value of an e4m3 byte: sign, 4 exponent bits (bias 7), 3 fraction bits; 0x7f and 0xff are NaN."""
    s, e, m = code >> 7, (code >> 3) & 15, code & 7
    if e == 15 and m == 7:
        return math.nan
    v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
    return -v if s else v


E4M3 = np.array([e4m3_value(c) for c in range(256)])
TOP = {"e4m3": 448.0, "i8": 127.0}


def pow2_scale(amax: float, code: str) -> float:
    """The smallest power of two s (at least 2^-126) with amax / s <= the largest code; 0 for amax = 0."""
    if amax == 0:
        return 0.0
    s = 2.0 ** -126
    while amax / s > TOP[code]:
        s *= 2
    return s


def encode(x, scale: float, code: str):
    """Codes (uint8) of x / scale: the nearest value, ties to the even code, saturated; 0 under scale 0."""
    x = np.asarray(x, dtype=np.float64)
    if scale == 0:
        return np.zeros(x.shape, dtype=np.uint8)
    y = np.clip(x / scale, -TOP[code], TOP[code])
    if code == "i8":
        return np.rint(y).astype(np.int64).astype(np.int8).view(np.uint8)
    mag = E4M3[:127]                                       # 0 .. 448, ascending with the code
    a = np.abs(y)
    hi = np.searchsorted(mag, a).clip(max=126)
    lo = np.maximum(hi - 1, 0)
    up = (mag[hi] - a < a - mag[lo]) | ((mag[hi] - a == a - mag[lo]) & (hi % 2 == 0))
    c = np.where(mag[hi] == a, hi, np.where(up, hi, lo))
    return (c + 128 * np.signbit(y)).astype(np.uint8)


def decode(codes, code: str):
    codes = np.asarray(codes, dtype=np.uint8)
    return codes.view(np.int8).astype(np.float64) if code == "i8" else E4M3[codes]


class BlockCache:
    """Codes uint8 [n_pages, heads, 64, d] for k and v, scales [n_pages, heads], means int8 [n_pages, heads, d]."""

    def __init__(self, k, v, k_scale, v_scale, mean, mean_scale, table, length, code):
        self.k, self.v = (np.array(a, dtype=np.uint8) for a in (k, v))
        self.k_scale, self.v_scale, self.mean_scale = (np.array(a, dtype=np.float64) for a in (k_scale, v_scale, mean_scale))
        self.mean, self.table, self.len, self.code = np.array(mean, dtype=np.int8), np.array(table), np.array(length), code

    def append(self, k, v, n_new):
        """k, v [B, heads, N, d]; one token after the other block, as the format defines it."""
        for b in range(len(self.len)):
            n0, m = int(self.len[b]), int(n_new[b])
            for j in range(n0 // BLOCK, -(-(n0 + m) // BLOCK) if m else 0):
                page = self.table[b, j]
                lo, hi = max(n0, j * BLOCK), min(n0 + m, (j + 1) * BLOCK)
                had, end = lo - j * BLOCK, hi - j * BLOCK
                for h in range(self.k.shape[1]):
                    for codes, scales, x in ((self.k, self.k_scale, k), (self.v, self.v_scale, v)):
                        new = np.asarray(x[b, h, lo - n0:hi - n0], dtype=np.float64)
                        start = scales[page, h] if had else 0.0
                        scale = max(start, pow2_scale(float(np.abs(new).max()), self.code))
                        if had and scale != start:
                            codes[page, h, :had] = encode(decode(codes[page, h, :had], self.code) * start, scale, self.code)
                        codes[page, h, had:end] = encode(new, scale, self.code)
                        scales[page, h] = scale
                    unit = 1.0 if self.code == "i8" else 2.0 ** -9
                    mean = decode(self.k[page, h, :end], self.code).sum(0) / unit / end
                    s = pow2_scale(float(np.abs(mean).max()), "i8")
                    self.mean[page, h] = encode(mean, s, "i8").view(np.int8)
                    self.mean_scale[page, h] = s * unit * self.k_scale[page, h]
            self.len[b] = n0 + m

    def tokens(self, b: int, h: int):
        """(k, v) [len, d] of a sequence and head, as the codes stand for."""
        n = int(self.len[b])
        pages = self.table[b, :-(-n // BLOCK)]
        k = decode(self.k[pages, h], self.code) * self.k_scale[pages, h][:, None, None]
        v = decode(self.v[pages, h], self.code) * self.v_scale[pages, h][:, None, None]
        return k.reshape(-1, k.shape[-1])[:n], v.reshape(-1, v.shape[-1])[:n]


def visible(length: int, Tq: int, t: int, causal: bool) -> int:
    """Keys that query t of Tq sees."""
    return max(length - Tq + 1 + t, 0) if causal else length


def select_blocks(cache: BlockCache, q, cap: int, first: int, last: int, causal: bool):
    """Lists [B][Tq][heads] of block indices, q [B, heads_q, Tq, d]; scores as exact fractions."""
    B, hq, Tq, d = q.shape
    heads = cache.k.shape[1]
    g = hq // heads
    out = np.empty((B, Tq, heads), dtype=object)
    for b in range(B):
        for t in range(Tq):
            for h in range(heads):
                nb = -(-visible(int(cache.len[b]), Tq, t, causal) // BLOCK)
                score = []
                for j in range(nb):
                    page = cache.table[b, j]
                    mean = cache.mean[page, h].astype(np.int64)
                    best = None
                    for e in range(g):
                        row = np.asarray(q[b, h * g + e, t], dtype=np.float64)
                        s = pow2_scale(float(np.abs(row).max()), "i8")
                        qi = encode(row, s, "i8").view(np.int8).astype(np.int64)
                        v = int(qi @ mean) * Fraction(s) * Fraction(float(cache.mean_scale[page, h]))
                        best = v if best is None or v > best else best
                    score.append((0 if j < first or j >= nb - last else 1, -best, j))
                out[b, t, h] = sorted(j for _, _, j in sorted(score)[:cap])
    return out


def cache_attention(cache: BlockCache, q, causal: bool, lists=None):
    """(o [B, heads_q, Tq, d], lse [B, heads_q, Tq]); lists as select_blocks gives them."""
    q = np.asarray(q, dtype=np.float64)
    B, hq, Tq, d = q.shape
    g = hq // cache.k.shape[1]
    o, lse = np.zeros(q.shape), np.full((B, hq, Tq), -np.inf)
    for b in range(B):
        for h in range(hq):
            k, v = cache.tokens(b, h // g)
            for t in range(Tq):
                see = np.arange(len(k)) < visible(len(k), Tq, t, causal)
                if lists is not None:
                    mine = np.zeros(-(-len(k) // BLOCK), dtype=bool)
                    mine[lists[b, t, h // g]] = True
                    see &= np.repeat(mine, BLOCK)[:len(k)]
                if not see.any():
                    continue
                s = k[see] @ q[b, h, t] / math.sqrt(d)
                m = s.max()
                p = np.exp(s - m)
                o[b, h, t] = p @ v[see] / p.sum()
                lse[b, h, t] = m + math.log(p.sum())
    return o, lse
