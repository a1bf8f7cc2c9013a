"""Reference of K/V held in 4 bits: the page format, the rounding of an append
and attention over such pools, from their definitions.

Shares no code with the library.
"""
from __future__ import annotations

import math

import numpy as np

from . import ref


def bf16_round(x) -> np.ndarray:
    """float32 values rounded to the nearest bf16 (ties to even), as float32;
    NaN stays NaN."""
    x = np.asarray(x, dtype=np.float32)
    b = x.view(np.uint32).astype(np.uint64)
    kept = ((b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
    return np.where(np.isnan(x), np.float32(np.nan), kept)


def quantize(x, group: int):
    """Groups of the last axis: (codes uint8 [.., D], step and origin float32
    [.., D / group]).  Differences and quotients are float32, as the rounding
    rules say; a group whose range is not finite is NaN, one whose step would be
    no normal bf16 has step 0 and every code 0."""
    x = np.asarray(x, dtype=np.float32)
    g = x.reshape(x.shape[:-1] + (-1, group))
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        lo, hi = g.min(-1), g.max(-1)
        span = hi - lo
        step, origin = bf16_round(span / np.float32(15)), bf16_round(lo)
        step = np.where(step < np.float32(2.0 ** -126), np.float32(0), step)
        bad = ~np.isfinite(span)
        step, origin = (np.where(bad, np.float32(np.nan), a) for a in (step, origin))
        q = (g - origin[..., None]) / step[..., None]
        code = np.where((step > 0)[..., None], np.clip(np.rint(q), 0, 15), 0)
    return code.astype(np.uint8).reshape(x.shape), step, origin


def dequantize(code, step, origin) -> np.ndarray:
    """float64 values of codes [.., D] under steps and origins [.., G]."""
    group = code.shape[-1] // step.shape[-1]
    s = np.repeat(np.asarray(step, np.float64), group, -1)
    z = np.repeat(np.asarray(origin, np.float64), group, -1)
    return z + s * code


def page_bytes(page_size, heads, dim, group) -> int:
    n = page_size * heads * (dim // 2) + page_size * heads * (dim // group) * 4
    return (n + 15) // 16 * 16


class Pool:
    """A K (or V) pool as bytes [pages, page_bytes], read and written row by row."""

    def __init__(self, data, page_size, heads, dim, group, layout):
        self.data, self.P, self.H, self.D, self.g = data, page_size, heads, dim, group
        self.layout = layout
        assert data.shape[-1] == page_bytes(page_size, heads, dim, group)

    @classmethod
    def empty(cls, pages, page_size, heads, dim, group, layout, fill=0):
        size = page_bytes(page_size, heads, dim, group)
        return cls(np.full((pages, size), fill, np.uint8), page_size, heads, dim, group, layout)

    def copy(self):
        return Pool(self.data.copy(), self.P, self.H, self.D, self.g, self.layout)

    def _row(self, slot, head):
        return slot * self.H + head if self.layout == "NHD" else head * self.P + slot

    def write(self, page, slot, rows):
        """rows [H, D] float32, quantised into a slot."""
        code, step, origin = quantize(rows, self.g)
        codes_end = self.P * self.H * (self.D // 2)
        for h in range(self.H):
            r = self._row(slot, h)
            packed = code[h, 0::2] | (code[h, 1::2] << 4)
            self.data[page, r * self.D // 2:(r + 1) * self.D // 2] = packed
            n = self.D // self.g * 4
            word = np.empty((self.D // self.g, 2), np.uint16)
            for i, a in enumerate((step[h], origin[h])):
                bits = a.view(np.uint32) >> 16
                word[:, i] = np.where(np.isnan(a), 0x7FC0, bits)
            self.data[page, codes_end + r * n:codes_end + (r + 1) * n] = \
                word.view(np.uint8).reshape(-1)

    def read(self, page, slot) -> np.ndarray:
        """[H, D] float64."""
        return self.rows(np.array([page]), np.array([slot]))[0]

    def rows(self, pages, slots) -> np.ndarray:
        """[n, H, D] float64 of the given slots."""
        h = np.arange(self.H)
        r = slots[:, None] * self.H + h if self.layout == "NHD" else h * self.P + slots[:, None]
        half = self.D // 2
        b = self.data[pages[:, None, None], r[..., None] * half + np.arange(half)]
        code = np.stack([b & 15, b >> 4], -1).reshape(b.shape[:-1] + (self.D,))
        n = self.D // self.g
        at = self.P * self.H * half + (r[..., None] * n + np.arange(n)) * 4

        def bf16_at(first):
            lo, hi = (self.data[pages[:, None, None], at + first + i].astype(np.uint16)
                      for i in (0, 1))
            return ref.bf16_bits_to_f64(lo | (hi << 8))

        return dequantize(code, bf16_at(0), bf16_at(2))


def fill(pool: Pool, kv_indptr, kv_indices, kv_lens, rows):
    """Write rows[r] [kv_len, H, D] into request r's slots."""
    for r, n in enumerate(kv_lens):
        for j in range(int(n)):
            page = int(kv_indices[int(kv_indptr[r]) + j // pool.P])
            pool.write(page, j % pool.P, rows[r][j])


def request_rows(pool: Pool, kv_indptr, kv_indices, r, n) -> np.ndarray:
    j = np.arange(n)
    pages = np.asarray(kv_indices)[int(kv_indptr[r]) + j // pool.P]
    return pool.rows(pages, j % pool.P)


def attention(q_bits, k_pool, v_pool, *, qo_indptr, kv_indptr, kv_indices, kv_lens, hq, hk,
              mask="causal", mask_bool=None, sm_scale=None):
    """(o, lse, a_k, a_v, a_2) float64: attention of q [rows, hq, D] (bf16 bits)
    over 4-bit pools.  a_k [rows, hq] bounds the magnitudes that a score sums, in
    log2 units, and a_v [rows, hq, D] those that an output sums, both by the
    parts (step * code and origin) that the words keep apart; a_2 [rows, hq] is
    the largest root of the sum of squares of a score's products."""
    q = ref.bf16_bits_to_f64(q_bits)
    d, g = q.shape[-1], hq // hk
    scale = sm_scale or 1.0 / math.sqrt(d)
    o, a_v = np.zeros(q.shape), np.zeros(q.shape)
    lse, a_k, a_2 = np.full(q.shape[:2], -np.inf), np.zeros(q.shape[:2]), np.zeros(q.shape[:2])
    at = 0
    k_parts, v_parts = _parts(k_pool), _parts(v_pool)
    for r, n in enumerate(kv_lens):
        n, q0, q1 = int(n), int(qo_indptr[r]), int(qo_indptr[r + 1])
        k, v, part_k, part_v = (request_rows(p, kv_indptr, kv_indices, r, n)
                                for p in (k_pool, v_pool, k_parts, v_parts))
        for i in range(q1 - q0):
            seen = np.ones(n, bool)
            if mask == "causal":
                seen = np.arange(n) <= n - (q1 - q0) + i
            elif mask == "custom":
                seen = np.asarray(mask_bool[at + i * n:at + (i + 1) * n], bool)
            if not seen.any():
                continue
            for h in range(hq):
                row, kh = q0 + i, h // g
                s = scale * (k[seen, kh] @ q[row, h])
                top = s.max()
                e = np.exp(s - top)
                o[row, h] = e @ v[seen, kh] / e.sum()
                lse[row, h] = (top + math.log(e.sum())) / math.log(2.0)
                log2 = scale / math.log(2.0)
                a_k[row, h] = log2 * (part_k[seen, kh] @ np.abs(q[row, h])).max()
                a_v[row, h] = e @ part_v[seen, kh] / e.sum()
                a_2[row, h] = log2 * math.sqrt(((k[seen, kh] ** 2) @ (q[row, h] ** 2)).max())
        at += (q1 - q0) * n
    return o, lse, a_k, a_v, a_2


def _parts(pool: Pool) -> Pool:
    """The pool of the magnitudes |step| * code + |origin|."""
    other = pool.copy()
    cut = pool.P * pool.H * (pool.D // 2)
    end = cut + pool.P * pool.H * (pool.D // pool.g) * 4
    other.data[:, cut + 1:end:2] &= 0x7F  # the sign bits of both halves of a word
    return other
