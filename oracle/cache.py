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


# ---------------------------------------------------------------------------
# The pages of the cache
# ---------------------------------------------------------------------------

def copy_pages(pool, src, dst, slots=None, *, layout="NHD"):
    """A copy of pool [..., pages, page, heads, dim] (HND: heads, page) with the
    first slots[i] slots of page src[i] written over those of page dst[i]."""
    out = np.array(pool, copy=True)
    axis = 0 if layout == "NHD" else 1
    for i in range(len(src)):
        n = None if slots is None else int(slots[i])
        part = (Ellipsis, int(src[i])), (Ellipsis, int(dst[i]))
        keep = (slice(None),) * axis + (slice(0, n),) + (slice(None),) * (2 - axis)
        out[part[1] + keep] = pool[part[0] + keep]
    return out


def alloc_pages(refs, n):
    """(page ids, new references): the n lowest pages without a reference."""
    refs, pages = list(refs), []
    for p, r in enumerate(refs):
        if r <= 0 and len(pages) < n:
            pages.append(p)
            refs[p] = 1
    if len(pages) < n:
        raise MemoryError("not enough free pages")
    return pages, refs


def free_pages(refs, pages):
    """References after one is dropped for each entry."""
    refs = list(refs)
    for p in pages:
        if not 0 <= p < len(refs) or refs[p] <= 0:
            raise ValueError("a reference that is not there")
        refs[p] -= 1
    return refs


def fork_pages(refs, tables, lens, page_size, parent, child_pages):
    """Tables of children.  tables / lens: page ids and token counts of the
    parents; parent: -1 or a parent's index; child_pages: pages of each child.
    Returns (child tables, copies [(src, dst, slots)], references)."""
    refs, out, copies = list(refs), [], []
    free = [p for p, r in enumerate(refs) if r <= 0][::-1]  # sharing frees none
    for p, n in zip(parent, child_pages):
        old = list(tables[p]) if p >= 0 else []
        partial = len(old) > 0 and lens[p] % page_size != 0
        shared = old[:len(old) - 1] if partial else old
        if n - len(shared) > len(free):
            raise MemoryError("not enough free pages")
        fresh = [free.pop() for _ in range(n - len(shared))]
        if partial:
            copies.append((old[-1], fresh[0], lens[p] % page_size))
        out.append(shared + fresh)
        for page in shared + fresh:
            refs[page] += 1
    return out, copies, refs


def compact_pages(refs, kv_indices):
    """(references, table entries, map, moves [(src, dst)], live pages) after
    the live pages moved to the front with the fewest moves."""
    live = [p for p, r in enumerate(refs) if r > 0]
    total = len(live)
    holes = [p for p in range(total) if refs[p] <= 0]
    movers = [p for p in reversed(live) if p >= total]
    moves = list(zip(movers, holes))
    to = {p: p for p in live if p < total} | dict(moves)
    new_refs = [0] * len(refs)
    for p, q in to.items():
        new_refs[q] = refs[p]
    return (new_refs, [to[p] for p in kv_indices], [to.get(p, -1) for p in range(len(refs))],
            moves, total)
