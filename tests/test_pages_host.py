"""The page operators without a GPU: what the entry points refuse before any
device work, and pins of the list-walking reference."""
import ctypes

import numpy as np
import pytest

import paged_kv_attention_plan_gb300 as pka
from oracle import cache
from paged_kv_attention_plan_gb300 import _pka

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 3, 4
A = 1 << 20  # an aligned address that a refused call never touches


def _copy(params=None, layers=2, k=A, v=A, stride=4096, layer=1 << 20, pages=9, src=A, dst=A,
          slots=A, n=3, count=A):
    params = params or pka.make_params(8, 2, 128, 16)
    return _pka.lib().pka_copy_pages(ctypes.byref(params), layers, k, v, stride, layer, pages, src,
                                     dst, slots, n, count, None)


@pytest.mark.parametrize("kw,want", [
    (dict(layers=-1), INVALID), (dict(n=-1), INVALID), (dict(pages=-1), INVALID),
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(src=None), INVALID),
    (dict(dst=None), INVALID), (dict(k=A + 8), INVALID), (dict(v=A + 2), INVALID),
    (dict(stride=0), INVALID), (dict(stride=4100), INVALID), (dict(layer=0), INVALID),
    (dict(layer=(1 << 20) + 4), INVALID), (dict(layers=40000), UNSUPPORTED), (dict(n=0), OK),
    (dict(layers=0), OK)])
def test_copy_refusals(kw, want):
    assert _copy(**kw) == want


def test_copy_refuses_bad_params():
    p = lambda **kw: pka.make_params(**{**dict(num_qo_heads=8, num_kv_heads=2, head_dim=128,  # noqa
                                               page_size=16), **kw})
    assert _copy(params=p(head_dim=80)) == UNSUPPORTED
    assert _copy(params=p(kv_ragged=True)) == UNSUPPORTED
    assert _copy(params=p(page_size=1 << 22)) == UNSUPPORTED
    assert _copy(params=p(page_size=0)) == INVALID
    assert _copy(params=p(kv_dtype="e4m3"), stride=4104) == INVALID


def _alloc(refs=A, pages=10, n=3, out=A):
    return _pka.lib().pka_alloc_pages(refs, pages, n, out, None)


@pytest.mark.parametrize("kw,want", [
    (dict(pages=-1), INVALID), (dict(n=-1), INVALID), (dict(n=11), WORKSPACE),
    (dict(refs=None), INVALID), (dict(out=None), INVALID), (dict(refs=A + 2), INVALID),
    (dict(n=0, refs=None, out=None), OK)])
def test_alloc_refusals(kw, want):
    assert _alloc(**kw) == want


@pytest.mark.parametrize("refs,pages,ids,n,want", [
    (A, -1, A, 3, INVALID), (A, 9, A, -3, INVALID), (None, 9, A, 3, INVALID),
    (A, 9, None, 3, INVALID), (A, 9, A + 1, 3, INVALID), (None, 9, None, 0, OK)])
def test_free_refusals(refs, pages, ids, n, want):
    assert _pka.lib().pka_free_pages(refs, pages, ids, n, None) == want


def _fork(P=4, refs=A, pages=10, parents=2, ptr=A, idx=A, n_idx=5, last=A, children=3, parent=A,
          child=A, table=2 * A, n_table=9, src=A, dst=A, slots=A, counts=A):
    return _pka.lib().pka_fork_pages(P, refs, pages, parents, ptr, idx, n_idx, last, children,
                                     parent, child, table, n_table, src, dst, slots, counts, None)


@pytest.mark.parametrize("kw,want", [
    (dict(P=0), INVALID), (dict(pages=-1), INVALID), (dict(parents=-1), INVALID),
    (dict(children=-1), INVALID), (dict(n_idx=-1), INVALID), (dict(n_table=-1), INVALID),
    (dict(children=8193), UNSUPPORTED), (dict(refs=None), INVALID), (dict(ptr=None), INVALID),
    (dict(idx=None), INVALID), (dict(last=None), INVALID), (dict(parent=None), INVALID),
    (dict(child=None), INVALID), (dict(table=None), INVALID), (dict(src=None), INVALID),
    (dict(dst=None), INVALID), (dict(slots=None), INVALID), (dict(counts=None), INVALID),
    (dict(table=A + 2), INVALID), (dict(counts=A + 1), INVALID),
    (dict(idx=2 * A), INVALID)])  # tables written over the parents' own
def test_fork_refusals(kw, want):
    assert _fork(**kw) == want


def _compact(refs=A, pages=10, idx=A, n=4, refs_out=A, idx_out=A, page_map=A, src=A, dst=A,
             counts=A):
    return _pka.lib().pka_compact_pages(refs, pages, idx, n, refs_out, idx_out, page_map, src,
                                        dst, counts, None)


@pytest.mark.parametrize("kw", [
    dict(pages=-1), dict(n=-1), dict(refs=None), dict(refs_out=None), dict(page_map=None),
    dict(src=None), dict(dst=None), dict(idx=None), dict(idx_out=None), dict(counts=None),
    dict(page_map=A + 2), dict(idx=A + 3)])
def test_compact_refusals(kw):
    assert _compact(**kw) == INVALID


# ---------------------------------------------------------------------------
# The reference
# ---------------------------------------------------------------------------

def test_reference_fork_worked_example():
    """Requests of 6 and 8 tokens in pages of 4: the first child of request 0
    shares page 7 and copies two slots of page 2; request 1's pages are full."""
    refs = [0, 0, 1, 1, 0, 1, 0, 1, 0]
    tables, copies, after = cache.fork_pages(refs, [[7, 2], [3, 5]], [6, 8], 4, [0, 1, -1],
                                             [2, 3, 1])
    assert tables == [[7, 0], [3, 5, 1], [4]]
    assert copies == [(2, 0, 2)]
    assert after == [1, 1, 1, 2, 1, 2, 0, 2, 0]


def test_reference_compact_worked_example():
    refs, table, page_map, moves, live = cache.compact_pages([0, 2, 0, 1, 0, 1], [1, 3, 5, 1])
    assert moves == [(5, 0), (3, 2)] and live == 3
    assert refs == [1, 2, 1, 0, 0, 0] and table == [1, 2, 0, 1]
    assert page_map == [-1, 1, -1, 2, -1, 0]


@pytest.mark.parametrize("seed", range(6))
def test_reference_compact_keeps_what_tables_read(seed):
    """Pages moved by the list and entries renamed: every entry reads what it read."""
    rng = np.random.default_rng(seed)
    n = int(rng.integers(2, 60))
    refs = (rng.random(n) < rng.random()) * rng.integers(1, 4, n)
    if not refs.any():
        refs[n - 1] = 1
    table = rng.choice(np.flatnonzero(refs), 40)
    pool = rng.standard_normal((n, 1, 1, 2))
    new_refs, new_table, page_map, moves, live = cache.compact_pages(refs, table)
    moved = cache.copy_pages(pool, [m[0] for m in moves], [m[1] for m in moves])
    assert np.array_equal(moved[new_table], pool[table])
    assert sorted(new_refs, reverse=True)[:live] == sorted(refs[refs > 0], reverse=True)
    assert all(r > 0 for r in new_refs[:live]) and not any(new_refs[live:])


def test_reference_alloc_and_free():
    pages, refs = cache.alloc_pages([1, 0, 2, 0, 0], 2)
    assert pages == [1, 3] and refs == [1, 1, 2, 1, 0]
    assert cache.free_pages(refs, [1, 2, 2]) == [1, 0, 0, 1, 0]
    with pytest.raises(MemoryError):
        cache.alloc_pages([1, 0], 2)
    with pytest.raises(ValueError):
        cache.free_pages([0, 1], [0])


def test_reference_copy_slots():
    x = np.arange(2 * 3 * 2 * 1, dtype=np.float64).reshape(2, 3, 2, 1)
    nhd = cache.copy_pages(x, [0], [1], [2])
    assert np.array_equal(nhd[1, :2], x[0, :2]) and np.array_equal(nhd[1, 2:], x[1, 2:])
    hnd = cache.copy_pages(x, [0], [1], [1], layout="HND")
    assert np.array_equal(hnd[1, :, :1], x[0, :, :1]) and np.array_equal(hnd[1, :, 1:], x[1, :, 1:])


@pytest.mark.parametrize("name", ["src", "dst", "slots", "count"])
@pytest.mark.parametrize("off", [1, 2, 3])
def test_copy_refuses_lists_off_their_alignment(name, off):
    """int32 arrays start at multiples of 4 bytes; the kernels could not read others."""
    assert _copy(**{name: A + off}) == INVALID


@pytest.mark.parametrize("table,n_table,idx,n_idx,refused", [
    (A, 8, A + 28, 5, True), (A + 16, 8, A, 5, True), (A + 8, 2, A, 50, True),
    (A, 50, A + 40, 1, True), (A, 8, A + 32, 5, False), (A + 20, 8, A, 5, False)])
def test_fork_refuses_tables_that_overlap(table, n_table, idx, n_idx, refused):
    """Children's tables written over any part of the parents'; tables that only
    meet go on to the next refusal, of the number of children."""
    status = _fork(table=table, n_table=n_table, idx=idx, n_idx=n_idx, children=8193)
    assert status == (INVALID if refused else UNSUPPORTED)
