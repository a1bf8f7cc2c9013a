"""Reference of the operators around the paged cache: rotary positions and
the append that rotates, in float64 and from their definitions.

Written for clarity, row by row; shares no code with the library.
"""
from __future__ import annotations

import numpy as np

from . import ref


def rope_frequencies(rotary_dim, base=10000.0, scaling="none", factor=1.0, original_len=0.0,
                     low_rotations=1.0, high_rotations=32.0):
    """Radians a position of each pair: base^(-2i/rotary_dim), divided by
    `factor` ("linear"), or blended between divided and kept by how often the
    pair turns over `original_len` positions ("parts")."""
    out = []
    for i in range(rotary_dim // 2):
        f = float(base) ** (-2.0 * i / rotary_dim)
        if scaling == "linear":
            f /= factor
        elif scaling == "parts":
            turns = original_len * f / (2 * np.pi)
            w = min(max((turns - low_rotations) / (high_rotations - low_rotations), 0.0), 1.0)
            f = (1 - w) * f / factor + w * f
        else:
            assert scaling == "none"
        out.append(f)
    return np.array(out)


def rope(x, positions, frequencies, *, interleaved=False, magnitude=1.0, transpose=False):
    """x [rows, heads, dim] float64 with its first 2 * len(frequencies)
    elements rotated to `positions`; transpose applies the transposed map."""
    x = np.asarray(x, dtype=np.float64)
    rd = 2 * len(frequencies)
    out = x.copy()
    # angle modulo one turn: float64 loses nothing that matters up to 2^31 positions
    t = np.asarray(positions, dtype=np.float64)[:, None] * frequencies[None, :]
    c, s = magnitude * np.cos(t)[:, None, :], magnitude * np.sin(t)[:, None, :]
    if transpose:
        s = -s
    i = np.arange(rd // 2)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + rd // 2)
    a, b = x[:, :, first], x[:, :, second]
    out[:, :, first] = a * c - b * s
    out[:, :, second] = a * s + b * c
    return out


def append_slots(append_indptr, kv_indptr, kv_indices, last_page_len, page_size):
    """(row, logical position, page, slot) of every appended row."""
    lens = ref.kv_lens_from_csr(kv_indptr, kv_indices, last_page_len, page_size)
    out = []
    for r, n in enumerate(lens):
        a0, a1 = int(append_indptr[r]), int(append_indptr[r + 1])
        pages = kv_indices[int(kv_indptr[r]):int(kv_indptr[r + 1])]
        for t in range(a1 - a0):
            pos = n - (a1 - a0) + t
            out.append((a0 + t, pos) + tuple(ref.token_address(pages, pos, page_size)))
    return out
