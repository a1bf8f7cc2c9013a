"""GPU parity of the page operators (copy, take, return, fork, compact) with
the reference that walks lists: whole numbers and moved bits, so all of it is
exact."""
import threading

import numpy as np
import pytest
import torch

import paged_kv_attention_plan_gb300 as pka
from inputs import workloads as W
from oracle import cache, ref
from tests.gpu_util import assert_parity, bf16, bits_of, f64, i32

pytestmark = pytest.mark.gpu

METADATA, WORKSPACE = 2, 4


def _host(*ts):
    torch.cuda.synchronize()
    out = [t.cpu().numpy() for t in ts]
    return out[0] if len(out) == 1 else out


def _refs(rng, n, live, most=4):
    refs = np.zeros(n, np.int32)
    held = rng.permutation(n)[:live]
    refs[held] = rng.integers(1, most, len(held))
    return refs


# ---------------------------------------------------------------------------
# Taking and returning
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("n", [1, 3, 127, 128, 129, 4096, 32771, 300001])
@pytest.mark.parametrize("live", [0.0, 0.5, 0.97])
@pytest.mark.parametrize("aligned", [True, False])
def test_alloc_takes_the_lowest(n, live, aligned):
    rng = np.random.default_rng(n)
    refs = _refs(rng, n, int(n * live))
    free = int((refs == 0).sum())
    for take in sorted({1, (free + 1) // 2, free}):
        d = i32(refs) if aligned else i32(np.concatenate([[7], refs]))[1:]
        pages = torch.full((take,), -9, dtype=torch.int32, device="cuda")
        pka.pka_alloc_pages(d, pages)
        got, after = _host(pages, d)
        want = np.flatnonzero(refs == 0)[:take]
        assert np.array_equal(got, want)
        refs_after = refs.copy()
        refs_after[want] = 1
        assert np.array_equal(after, refs_after)
    assert pka.pka_get_device_error() == 0


def test_alloc_matches_the_list_walk():
    rng = np.random.default_rng(0)
    refs = _refs(rng, 500, 200)
    d, pages = i32(refs), torch.empty(77, dtype=torch.int32, device="cuda")
    pka.pka_alloc_pages(d, pages)
    want, after = cache.alloc_pages(refs, 77)
    assert np.array_equal(_host(pages), want) and np.array_equal(_host(d), after)


def test_alloc_with_too_few_free_takes_none():
    rng = np.random.default_rng(1)
    refs = _refs(rng, 5000, 4000)
    d, pages = i32(refs), torch.full((1001,), 5, dtype=torch.int32, device="cuda")
    pka.pka_alloc_pages(d, pages)
    assert np.all(_host(pages) == -1) and np.array_equal(_host(d), refs)
    assert pka.pka_get_device_error() == WORKSPACE
    with pytest.raises(pka.PkaError) as e:
        pka.pka_alloc_pages(d, torch.empty(5001, dtype=torch.int32, device="cuda"))
    assert e.value.status == WORKSPACE
    pka.pka_alloc_pages(d, pages[:0])
    assert np.array_equal(_host(d), refs) and pka.pka_get_device_error() == 0


@pytest.mark.parametrize("n", [1, 31, 1000, 200003])
def test_free_drops_one_reference_an_entry(n):
    rng = np.random.default_rng(n)
    refs = _refs(rng, n, (n + 1) // 2, 5)
    entries = np.repeat(np.arange(n), refs)  # every reference once
    entries = rng.permutation(entries)[:max(1, len(entries) * 2 // 3)].astype(np.int32)
    d = i32(refs)
    pka.pka_free_pages(d, i32(entries))
    assert np.array_equal(_host(d), cache.free_pages(refs, entries))
    assert pka.pka_get_device_error() == 0


def test_free_of_what_is_not_held_is_skipped_and_noted():
    refs = np.array([2, 0, 1, 3], np.int32)
    for entries, after in (([0, 0, 0, 0, 2], [0, 0, 0, 3]), ([1, 1, 3], [2, 0, 1, 2]),
                           ([-1, 4, 1 << 30, 2], [2, 0, 0, 3])):
        d = i32(refs)
        pka.pka_free_pages(d, i32(entries))
        assert np.array_equal(_host(d), after)
        assert pka.pka_get_device_error() == METADATA
    d = i32([3])
    pka.pka_free_pages(d, i32([0] * 5000))  # many more than there are, at once
    assert np.array_equal(_host(d), [0]) and pka.pka_get_device_error() == METADATA


# ---------------------------------------------------------------------------
# Fork
# ---------------------------------------------------------------------------

def _parents(rng, lens, page, pool):
    pages = -(-np.asarray(lens) // page)
    indptr = np.concatenate([[0], np.cumsum(pages)]).astype(np.int32)
    ids = rng.permutation(pool)[:indptr[-1]].astype(np.int32)
    last = np.where(pages > 0, lens - (pages - 1) * page, 1).astype(np.int32)
    return indptr, ids, last


def _fork(page, refs, indptr, ids, last, parent, child_pages, room=0):
    child = np.concatenate([[0], np.cumsum(child_pages)]).astype(np.int32)
    n = len(parent)
    d = dict(refs=i32(refs), table=torch.full((int(child[-1]) + room,), -5, dtype=torch.int32,
                                              device="cuda"),
             counts=torch.full((2,), -5, dtype=torch.int32, device="cuda"))
    for name in ("src", "dst", "slots"):
        d[name] = torch.full((n,), -5, dtype=torch.int32, device="cuda")
    pka.pka_fork_pages(page, d["refs"], i32(indptr), i32(ids), i32(last), i32(parent), i32(child),
                       d["table"], d["src"], d["dst"], d["slots"], d["counts"])
    torch.cuda.synchronize()
    return child, {k: v.cpu().numpy() for k, v in d.items()}


def _check_fork(page, refs, lens, indptr, ids, last, parent, child_pages, room=0):
    child, got = _fork(page, refs, indptr, ids, last, parent, child_pages, room)
    tables = [ids[indptr[r]:indptr[r + 1]].tolist() for r in range(len(lens))]
    want, copies, refs_after = cache.fork_pages(refs, tables, lens, page, parent, child_pages)
    for c, t in enumerate(want):
        assert np.array_equal(got["table"][child[c]:child[c + 1]], t)
    assert np.all(got["table"][child[-1]:] == -5)
    assert np.array_equal(got["refs"], refs_after)
    n = len(copies)
    assert np.array_equal(np.stack([got["src"], got["dst"], got["slots"]], 1)[:n],
                          np.array(copies, np.int32).reshape(n, 3))
    assert all(np.all(got[k][n:] == -5) for k in ("src", "dst", "slots"))
    assert got["counts"][0] == n
    assert got["counts"][1] == int(((np.asarray(refs_after) > 0) & (np.asarray(refs) <= 0)).sum())
    assert pka.pka_get_device_error() == 0


@pytest.mark.parametrize("page", [1, 4, 16])
@pytest.mark.parametrize("children", [1, 7, 33, 1100, 8192])
def test_fork_matches_the_list_walk(page, children):
    rng = np.random.default_rng(page * children)
    n = min(children, 9)
    lens = rng.integers(1, 60, n)
    lens[0] = 4 * page  # a full last page
    if n > 2:
        lens[1] = 0  # a parent without pages
    pool = int(2000 + children * (60 // page + 4))
    indptr, ids, last = _parents(rng, lens, page, pool)
    refs = np.zeros(pool, np.int32)
    refs[ids] = 1
    refs[rng.permutation(pool)[:300]] += 1  # pages that others hold
    parent = rng.integers(-1, n, children).astype(np.int32)
    pages = indptr[1:] - indptr[:-1]
    grown = np.where(parent >= 0, pages[np.maximum(parent, 0)], 0) + rng.integers(0, 3, children)
    _check_fork(page, refs, lens, indptr, ids, last, parent, grown, room=5)


def test_fork_one_prompt_into_samples():
    rng = np.random.default_rng(4)
    lens = np.array([2040])
    indptr, ids, last = _parents(rng, lens, 16, 1000)
    refs = np.zeros(1000, np.int32)
    refs[ids] = 1
    _check_fork(16, refs, lens, indptr, ids, last, np.zeros(8, np.int32), np.full(8, 129))
    _check_fork(16, refs, lens, indptr, ids, last, np.zeros(1, np.int32), np.full(1, 128))


def test_fork_beams_with_long_tables():
    rng = np.random.default_rng(5)
    lens = rng.integers(3000, 6000, 16)
    indptr, ids, last = _parents(rng, lens, 1, 200000)
    refs = np.zeros(200000, np.int32)
    refs[ids] = 1
    parent = rng.integers(0, 16, 64).astype(np.int32)
    _check_fork(1, refs, lens, indptr, ids, last, parent, lens[parent] + 1)


@pytest.mark.parametrize("children", [700, 1500])
def test_fork_long_and_short_tables_together(children):
    """Tables of one page beside tables of hundreds and tens of thousands, in
    any order, around the lengths (255..257 shared pages) and counts where the
    references of long tables are added together."""
    rng = np.random.default_rng(children)
    lens = np.array([1, 255, 256, 257, 700, 1, 3, 40000])
    indptr, ids, last = _parents(rng, lens, 1, 400000)
    refs = np.zeros(400000, np.int32)
    refs[ids] = 1
    parent = rng.choice([-1, 0, 1, 2, 3, 4, 5, 6], children).astype(np.int32)
    parent[[3, 4, 650]] = 7
    grown = np.where(parent >= 0, lens[np.maximum(parent, 0)], 0) + rng.integers(0, 2, children)
    _check_fork(1, refs, lens, indptr, ids, last, parent, grown)


def test_fork_with_every_page_taken():
    """Exactly as many free pages as needed, then one fewer."""
    rng = np.random.default_rng(6)
    lens = np.array([10, 6])
    indptr, ids, last = _parents(rng, lens, 4, 12)  # 3 + 2 pages, both partial
    refs = np.ones(12, np.int32)
    for p in [p for p in range(12) if p not in ids][:4]:
        refs[p] = 0
    _check_fork(4, refs, lens, indptr, ids, last, np.array([0, 1, 0], np.int32), [3, 3, 3])
    _, got = _fork(4, refs, indptr, ids, last, np.array([0, 1, 0], np.int32), [3, 3, 4])
    _refused(got, refs, WORKSPACE)


def _refused(got, refs, status):
    assert np.array_equal(got["refs"], refs)
    assert got["counts"].tolist() == [-1, -1]
    assert all(np.all(got[k] == -5) for k in ("table", "src", "dst", "slots"))
    assert pka.pka_get_device_error() == status


@pytest.mark.parametrize("what", ["parent_high", "parent_low", "short", "decreasing", "past_end",
                                  "last_zero", "last_high", "indptr", "indptr_past"])
def test_fork_refuses_malformed_arrays(what):
    rng = np.random.default_rng(7)
    lens = np.array([9, 5, 12])
    indptr, ids, last = _parents(rng, lens, 4, 40)
    refs = np.zeros(40, np.int32)
    refs[ids] = 1
    parent, pages = np.array([0, 1, 2, 0, -1], np.int32), np.array([3, 3, 3, 4, 2])
    if what == "parent_high":
        parent[2] = 3
    if what == "parent_low":
        parent[2] = -2
    if what == "short":
        pages[3] = 2
    if what == "decreasing":
        pages[4] = -1
    if what == "last_zero":
        last[1] = 0
    if what == "last_high":
        last[1] = 5
    if what == "indptr":
        indptr[1], indptr[2] = indptr[2], indptr[1]
    if what == "indptr_past":
        indptr[3] = 999
    _, got = _fork(4, refs, indptr, ids, last, parent, pages, room=-1 if what == "past_end" else 9)
    _refused(got, refs, METADATA)


def test_fork_carries_a_bad_page_over_and_notes_it():
    rng = np.random.default_rng(8)
    lens = np.array([16])
    indptr, ids, last = _parents(rng, lens, 4, 20)
    refs = np.zeros(20, np.int32)
    refs[ids] = 1
    ids[1] = 77
    _, got = _fork(4, refs, indptr, ids, last, np.zeros(2, np.int32), [4, 4])
    assert got["table"].tolist() == ids.tolist() * 2
    after = refs.copy()
    after[ids[[0, 2, 3]]] += 2
    assert np.array_equal(got["refs"], after)
    assert pka.pka_get_device_error() == METADATA


@pytest.mark.parametrize("length,children", [(40, 6), (900, 30)])
def test_fork_of_parents_that_share_pages(length, children):
    """Parents with a common prefix (already forked once), one page listed twice
    in a table: every entry of every child is one reference more."""
    rng = np.random.default_rng(length)
    pool = 20 * length
    lens = np.array([length, length, length + 3])
    indptr, ids, last = _parents(rng, lens, 1, pool)
    ids[indptr[1]:indptr[1] + length // 2] = ids[:length // 2]
    ids[indptr[2]:indptr[2] + length // 3] = ids[:length // 3]
    ids[indptr[2] + length // 3] = ids[0]
    refs = np.bincount(ids, minlength=pool).astype(np.int32)
    parent = rng.integers(0, 3, children).astype(np.int32)
    _check_fork(1, refs, lens, indptr, ids, last, parent, lens[parent] + 2)


def test_fork_of_nothing():
    refs = i32([1, 0])
    empty = torch.empty(0, dtype=torch.int32, device="cuda")
    counts = i32([5, 5])
    pka.pka_fork_pages(4, refs, i32([0, 1]), i32([0]), i32([2]), empty, i32([0]), empty, empty,
                       empty, empty, counts)
    assert _host(counts).tolist() == [0, 0] and _host(refs).tolist() == [1, 0]
    # children without pages
    one = torch.full((2,), -5, dtype=torch.int32, device="cuda")
    pka.pka_fork_pages(4, refs, i32([0, 1]), i32([0]), i32([2]), i32([-1, -1]), i32([0, 0, 0]),
                       empty, one, one, one, counts)
    assert _host(counts).tolist() == [0, 0] and _host(refs).tolist() == [1, 0]
    assert pka.pka_get_device_error() == 0


# ---------------------------------------------------------------------------
# Compact
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("n", [1, 2, 5, 127, 128, 130, 5000, 32769, 250007])
@pytest.mark.parametrize("live", [0.0, 0.3, 0.9, 1.0])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact_matches_the_list_walk(n, live, in_place):
    rng = np.random.default_rng(n)
    refs = _refs(rng, n, int(round(n * live)))
    held = np.flatnonzero(refs)
    idx = rng.choice(held, 2 * n).astype(np.int32) if len(held) else np.zeros(0, np.int32)
    d, t = i32(refs), i32(idx)
    d_out, t_out = (d, t) if in_place else (torch.full_like(d, -5), torch.full_like(t, -5))
    page_map = torch.full_like(d, -5)
    src, dst = (torch.full((n // 2,), -5, dtype=torch.int32, device="cuda") for _ in range(2))
    counts = torch.full((2,), -5, dtype=torch.int32, device="cuda")
    pka.pka_compact_pages(d, t, d_out, t_out, page_map, src, dst, counts)
    want_refs, want_idx, want_map, moves, total = cache.compact_pages(refs, idx)
    assert np.array_equal(_host(d_out), want_refs)
    assert np.array_equal(_host(t_out), want_idx)
    assert np.array_equal(_host(page_map), want_map)
    m = len(moves)
    assert _host(counts).tolist() == [m, total]
    got = np.stack(_host(src, dst), 1)
    assert np.array_equal(got[:m], np.array(moves, np.int32).reshape(m, 2))
    assert np.all(got[m:] == -5)
    if not in_place:
        assert np.array_equal(_host(d), refs) and np.array_equal(_host(t), idx)
    assert pka.pka_get_device_error() == 0


@pytest.mark.parametrize("n", [700, 300_001])
def test_arrays_at_any_4_byte_address(n):
    """Arrays that start 4, 8 and 12 bytes past a 16-byte boundary."""
    rng = np.random.default_rng(n)
    refs = _refs(rng, n, n // 2)

    def off(a, by):
        return i32(np.concatenate([np.full(by, -77), a]))[by:]

    for by in (1, 2, 3):
        d, out, page_map = off(refs, by), off(np.zeros(n), by), off(np.zeros(n), 4 - by)
        table = off(np.flatnonzero(refs), by)
        src, dst = (off(np.zeros(n // 2), by) for _ in range(2))
        counts = off(np.zeros(2), by)
        pka.pka_compact_pages(d, table, out, table, page_map, src, dst, counts)
        w_refs, w_to, w_map, moves, live = cache.compact_pages(refs, np.flatnonzero(refs))
        assert np.array_equal(_host(out), w_refs) and np.array_equal(_host(table), w_to)
        assert np.array_equal(_host(page_map), w_map)
        assert _host(counts).tolist() == [len(moves), live]
        assert np.array_equal(np.stack(_host(src, dst), 1)[:len(moves)],
                              np.array(moves, np.int32).reshape(-1, 2))
        pages = off(np.zeros(n // 3), by)
        pka.pka_alloc_pages(d, pages)
        want = np.flatnonzero(refs == 0)[:n // 3]
        assert np.array_equal(_host(pages), want)
        pka.pka_free_pages(d, pages)
        assert np.array_equal(_host(d), refs)
    assert pka.pka_get_device_error() == 0


def test_compact_of_an_empty_pool():
    empty, t = torch.empty(0, dtype=torch.int32, device="cuda"), i32([0, 4])
    counts = i32([5, 5])
    pka.pka_compact_pages(empty, t, empty, t, empty, empty, empty, counts)
    assert _host(counts).tolist() == [0, 0] and _host(t).tolist() == [0, 4]
    assert pka.pka_get_device_error() == METADATA
    pka.pka_compact_pages(empty, empty, empty, empty, empty, empty, empty, counts)
    assert pka.pka_get_device_error() == 0


def test_compact_leaves_and_notes_entries_of_no_live_page():
    refs = np.array([0, 2, 0, 1, 0, 1], np.int32)
    d, t = i32(refs), i32([1, 3, 0, -4, 6, 5])
    page_map, counts = torch.empty_like(d), torch.empty(2, dtype=torch.int32, device="cuda")
    src, dst = (torch.empty(3, dtype=torch.int32, device="cuda") for _ in range(2))
    pka.pka_compact_pages(d, t, d, t, page_map, src, dst, counts)
    # live 1, 3, 5 -> 5 to 0, 3 to 2
    assert _host(t).tolist() == [1, 2, 0, -4, 6, 0] and _host(d).tolist() == [1, 2, 1, 0, 0, 0]
    assert _host(counts).tolist() == [2, 3]
    assert pka.pka_get_device_error() == METADATA


# ---------------------------------------------------------------------------
# Copy
# ---------------------------------------------------------------------------

def _pool(rng, kv, shape):
    return (W.e4m3_codes(rng, shape) if kv == "e4m3" else W.normal_bf16_bits(rng, shape))


def _dev(x):
    return torch.from_numpy(x.copy()).cuda() if x.dtype == np.uint8 else bf16(x)


def _back(t):
    torch.cuda.synchronize()
    return t.cpu().numpy() if t.dtype == torch.uint8 else bits_of(t)


@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("page,hk,d", [(1, 1, 64), (1, 8, 128), (3, 5, 64), (4, 2, 128),
                                       (16, 8, 128), (64, 3, 64)])
@pytest.mark.parametrize("partial", [False, True])
def test_copy_bits(layout, kv, page, hk, d, partial):
    rng = np.random.default_rng(page + hk)
    layers, pages, n = 3, 23, 9
    shape = (layers, pages, 2) + ((page, hk) if layout == "NHD" else (hk, page)) + (d,)
    x = _pool(rng, kv, shape)
    ids = rng.permutation(pages).astype(np.int32)
    src, dst = ids[:n], ids[n:2 * n]
    slots = rng.integers(0, page + 1, n).astype(np.int32) if partial else None
    params = pka.make_params(hk, hk, d, page, layout, kv_dtype=kv)
    t = _dev(x)
    pka.pka_copy_pages(params, t[:, :, 0], t[:, :, 1], i32(src), i32(dst),
                       None if slots is None else i32(slots))
    got = _back(t)
    for w in range(2):
        assert np.array_equal(got[:, :, w], cache.copy_pages(x[:, :, w], src, dst, slots,
                                                             layout=layout))
    # one layer, K and V apart
    k, v = _dev(x[1, :, 0]), _dev(x[1, :, 1])
    pka.pka_copy_pages(params, k, v, i32(src), i32(dst), None if slots is None else i32(slots))
    assert np.array_equal(_back(k), got[1, :, 0]) and np.array_equal(_back(v), got[1, :, 1])
    assert pka.pka_get_device_error() == 0


def test_copy_counts_from_the_device_and_skips():
    rng = np.random.default_rng(2)
    x = _pool(rng, "bf16", (2, 12, 2, 4, 2, 64))
    params = pka.make_params(2, 2, 64, 4)
    src, dst = np.array([0, 1, 2, 3], np.int32), np.array([8, 9, 10, 11], np.int32)

    def run(src, dst, count=None, slots=None):
        t = _dev(x)
        pka.pka_copy_pages(params, t[:, :, 0], t[:, :, 1], i32(src), i32(dst),
                           None if slots is None else i32(slots),
                           None if count is None else i32([count, 77]))
        return _back(t)

    def want(src, dst, slots=None):
        return np.stack([cache.copy_pages(x[:, :, w], src, dst, slots) for w in range(2)], 2)

    for count, n in ((0, 0), (-1, 0), (3, 3), (4, 4), (99, 4)):
        assert np.array_equal(run(src, dst, count), want(src[:n], dst[:n]))
    assert np.array_equal(run(src[:0], dst[:0]), x)
    assert np.array_equal(run([0, 5], [0, 6]), want([5], [6]))  # a page onto itself
    assert pka.pka_get_device_error() == 0
    assert np.array_equal(run([0, -1, 12, 3, 4], [8, 9, 10, -1, 1 << 30]), want([0], [8]))
    assert pka.pka_get_device_error() == METADATA
    assert np.array_equal(run(src, dst, slots=[4, -1, 5, 2]), want([0, 3], [8, 11], [4, 2]))
    assert pka.pka_get_device_error() == METADATA


def test_binding_refuses_what_it_cannot_pass(monkeypatch):
    """Shapes, types, layouts and devices that never reach the library."""
    def t(*shape, dtype=torch.int32):
        return torch.zeros(*shape, dtype=dtype, device="cuda")
    bf = torch.bfloat16
    params, rope = pka.make_params(2, 2, 64, 4), pka.make_rope(64)
    k, ids, q = t(3, 5, 4, 2, 64, dtype=bf), t(2), t(6, 2, 64, dtype=bf)
    calls = [
        (ValueError, lambda: pka.pka_copy_pages(params, k, k[:, :4], ids, ids)),
        (ValueError, lambda: pka.pka_copy_pages(params, k, k, ids, t(3))),
        (ValueError, lambda: pka.pka_copy_pages(params, k.transpose(2, 3), k.transpose(2, 3), ids,
                                                ids)),
        (TypeError, lambda: pka.pka_copy_pages(params, k.float(), k.float(), ids, ids)),
        (TypeError, lambda: pka.pka_copy_pages(params, k, k, ids.long(), ids.long())),
        (TypeError, lambda: pka.pka_copy_pages(params, k.cpu(), k.cpu(), ids, ids)),
        (TypeError, lambda: pka.pka_alloc_pages(t(4).cpu(), ids)),
        (ValueError, lambda: pka.pka_alloc_pages(t(8)[::2], ids)),
        (ValueError, lambda: pka.pka_fork_pages(4, t(9), t(2), t(3), t(2), ids, t(3), t(4), ids,
                                                ids, ids, t(2))),
        (ValueError, lambda: pka.pka_fork_pages(4, t(9), t(2), t(3), t(1), ids, t(3), t(4), t(1),
                                                ids, ids, t(2))),
        (ValueError, lambda: pka.pka_compact_pages(t(9), t(3), t(8), t(3), t(9), t(4), t(4), t(2))),
        (ValueError, lambda: pka.pka_compact_pages(t(9), t(3), t(9), t(3), t(9), t(3), t(4), t(2))),
        (ValueError, lambda: pka.pka_apply_rope(rope, t(6))),
        (ValueError, lambda: pka.pka_apply_rope(rope, t(5), q, q)),
        (ValueError, lambda: pka.pka_apply_rope(rope, t(6), q, t(6, 3, 64, dtype=bf))),
        (ValueError, lambda: pka.pka_apply_rope(rope, t(6), q.transpose(0, 1), q)),
        (TypeError, lambda: pka.pka_apply_rope(rope, t(6), q.half(), q)),
        (TypeError, lambda: pka.pka_apply_rope(rope, t(6), q, None)),
        (ValueError, lambda: pka.pka_rope_append_paged_kv_cache(
            params, rope, None, None, q, q, t(3), t(2), t(1), t(1), k[0], k[1], k.stride(1))),
    ]
    for error, call in calls:
        with pytest.raises(error):
            call()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for call in (lambda: pka.pka_free_pages(t(4), ids),
                 lambda: pka.pka_apply_rope(rope, t(6), q, q),
                 lambda: pka.pka_copy_pages(params, k, k, ids, ids)):
        with pytest.raises(ValueError, match="current device"):
            call()


def test_copy_and_append_past_32_bit_offsets():
    """Pages whose byte and element offsets pass 2^32, in one allocation of K
    and V (9.2 GB)."""
    pages, page, hk, d = 140_000, 16, 8, 128
    t = torch.empty(pages, 2, page, hk, d, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(3)
    x = _pool(rng, "bf16", (3, 2, page, hk, d))
    low, high = [5, 6, 7], [pages - 1, pages - 2, 70_001]
    t[torch.tensor(low)] = bf16(x)
    params = pka.make_params(hk, hk, d, page)
    k, v = t[:, 0], t[:, 1]
    pka.pka_copy_pages(params, k, v, i32(low), i32(high))
    torch.cuda.synchronize()
    assert np.array_equal(bits_of(t[torch.tensor(high).cuda()]), x)
    # 20 rows appended over the last two pages of the pool
    new = W.normal_bf16_bits(rng, (20, hk, d))
    pka.pka_rope_append_paged_kv_cache(params, pka.make_rope(128), None, None, bf16(new),
                                       bf16(new), i32([0, 20]), i32([0, 2]),
                                       i32([pages - 2, pages - 1]), i32([4]), k, v, k.stride(0))
    torch.cuda.synchronize()
    assert np.array_equal(bits_of(t[pages - 2, 1]), new[:16])
    got = bits_of(t[pages - 1, 1])
    assert np.array_equal(got[:4], new[16:]) and np.array_equal(got[4:], x[0, 1, 4:])
    assert pka.pka_get_device_error() == 0


# ---------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("layout,page,kv", [("NHD", 16, "bf16"), ("HND", 4, "bf16"),
                                            ("NHD", 1, "bf16"), ("HND", 16, "e4m3")])
def test_fork_append_attend_return_compact_attend(layout, page, kv):
    """Two prompts fork into five requests, each appends its own rotated token
    and attends; the prompts are returned, the pool is compacted, and the same
    attention over the moved pages gives the same bits."""
    rng = np.random.default_rng(page)
    hq, hk, d, pool = 8, 2, 128, 400
    lens = np.array([70, 33])
    indptr, ids, last = _parents(rng, lens, page, pool)
    refs = np.zeros(pool, np.int32)
    refs[ids] = 1
    shape = (pool, 2) + ((page, hk) if layout == "NHD" else (hk, page)) + (d,)
    x = _pool(rng, kv, shape)
    parent = np.array([0, 1, 0, 0, 1], np.int32)
    new_lens = lens[parent] + 1
    child_pages = -(-new_lens // page)
    child = np.concatenate([[0], np.cumsum(child_pages)]).astype(np.int32)
    child_last = (new_lens - (child_pages - 1) * page).astype(np.int32)
    scales = (0.5, 0.25) if kv == "e4m3" else (1.0, 1.0)
    params = pka.make_params(hq, hk, d, page, layout, kv_dtype=kv, k_scale=scales[0],
                             v_scale=scales[1])
    t, r = _dev(x), i32(refs)
    k, v = t[:, 0], t[:, 1]
    table = torch.empty(int(child[-1]), dtype=torch.int32, device="cuda")
    src, dst, slots = (torch.empty(5, dtype=torch.int32, device="cuda") for _ in range(3))
    counts = torch.empty(2, dtype=torch.int32, device="cuda")
    child_ptr, child_last_d = i32(child), i32(child_last)
    pka.pka_fork_pages(page, r, i32(indptr), i32(ids), i32(last), i32(parent), child_ptr, table,
                       src, dst, slots, counts)
    pka.pka_copy_pages(params, k, v, src, dst, slots, counts)
    q, k_new, v_new = (W.normal_bf16_bits(rng, (5, h, d)) for h in (hq, hk, hk))
    rope, freqs = pka.make_rope(d), cache.rope_frequencies(d)
    qd = bf16(q)
    app = i32(np.arange(6))
    pka.pka_rope_append_paged_kv_cache(params, rope, qd, qd, bf16(k_new), bf16(v_new), app,
                                       child_ptr, table, child_last_d, k, v, k.stride(0))
    attn = pka.BatchAttention()
    attn.plan(None, child, child_last, num_qo_heads=hq, num_kv_heads=hk, head_dim=d,
              page_size=page, layout=layout, kv_dtype=kv, k_scale=scales[0], v_scale=scales[1])
    o, lse = attn.run(qd, k, v, table)
    torch.cuda.synchronize()
    assert pka.pka_get_device_error() == 0
    # the oracle: every child's history by the parent's own pages, its token behind it
    tables = [ids[indptr[i]:indptr[i + 1]] for i in range(2)]
    where = cache.append_slots(np.arange(6), child, table.cpu().numpy(), child_last, page)
    pos = np.array([w[1] for w in where])
    assert np.array_equal(pos, lens[parent])
    bits = _back(t)
    swap = (lambda y: y) if layout == "NHD" else (lambda y: y.transpose(0, 2, 1, 3))
    kb, vb = swap(bits[:, 0]), swap(bits[:, 1])
    xk, xv = swap(x[:, 0]), swap(x[:, 1])
    for c in range(5):
        old = tables[parent[c]]
        new = table.cpu().numpy()[child[c]:child[c + 1]]
        for j in range(lens[parent[c]]):
            assert np.array_equal(kb[new[j // page], j % page], xk[old[j // page], j % page])
            assert np.array_equal(vb[new[j // page], j % page], xv[old[j // page], j % page])
    o_ref, lse_ref = ref.batch_attention(
        bits_of(qd), bits[:, 0], bits[:, 1], qo_indptr=np.arange(6, dtype=np.int32),
        kv_indptr=child, kv_indices=table.cpu().numpy(), last_page_len=child_last, page_size=page,
        num_qo_heads=hq, num_kv_heads=hk, layout=layout, kv_dtype=kv, k_scale=scales[0],
        v_scale=scales[1])
    assert_parity(f64(o), f64(lse), o_ref, lse_ref)
    rotated = cache.rope(ref.bf16_bits_to_f64(q), pos, freqs)
    assert np.abs(ref.bf16_bits_to_f64(bits_of(qd)) - rotated).max() <= 2.0 ** -8 * np.abs(
        rotated).max() + 1e-4
    # return the prompts, move what is left to the front, attend again
    pka.pka_free_pages(r, i32(ids))
    before = _host(r).copy()
    assert before.sum() == len(table)
    page_map = torch.empty_like(r)
    cs, cd = (torch.empty(pool // 2, dtype=torch.int32, device="cuda") for _ in range(2))
    pka.pka_compact_pages(r, table, r, table, page_map, cs, cd, counts)
    pka.pka_copy_pages(params, k, v, cs, cd, None, counts)
    o2, lse2 = attn.run(qd, k, v, table)
    torch.cuda.synchronize()
    live = int((before > 0).sum())
    assert _host(counts)[1] == live and int(table.max()) < live
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    pka.pka_free_pages(r, table)
    assert not _host(r).any()
    assert pka.pka_get_device_error() == 0


def test_calls_at_once_on_streams_and_graphs():
    """Takes and compactions of two pools at the same time, on two streams and
    from two captured graphs: no call keeps anything another could meet."""
    rng = np.random.default_rng(13)
    pools = [_refs(rng, n, n // 2) for n in (300_000, 400_000)]
    work = []
    for refs in pools:
        r = i32(refs)
        d = dict(r=r, pages=torch.empty(100_000, dtype=torch.int32, device="cuda"),
                 out=torch.empty_like(r), table=i32(np.flatnonzero(refs)),
                 map=torch.empty_like(r), counts=i32([0, 0]), stream=torch.cuda.Stream())
        d["to"] = torch.empty_like(d["table"])
        d["src"], d["dst"] = (torch.empty(len(refs) // 2, dtype=torch.int32, device="cuda")
                              for _ in range(2))
        work.append(d)

    def step(d):
        pka.pka_alloc_pages(d["r"], d["pages"], stream=d["stream"])
        pka.pka_free_pages(d["r"], d["pages"], stream=d["stream"])
        pka.pka_compact_pages(d["r"], d["table"], d["out"], d["to"], d["map"], d["src"], d["dst"],
                              d["counts"], stream=d["stream"])

    def check():
        torch.cuda.synchronize()
        for refs, d in zip(pools, work):
            assert np.array_equal(_host(d["r"]), refs)
            assert np.array_equal(_host(d["pages"]), np.flatnonzero(refs == 0)[:100_000])
            w_refs, w_to, w_map, moves, live = cache.compact_pages(refs, np.flatnonzero(refs))
            assert np.array_equal(_host(d["out"]), w_refs)
            assert np.array_equal(_host(d["to"]), w_to) and np.array_equal(_host(d["map"]), w_map)
            assert _host(d["counts"]).tolist() == [len(moves), live]
            for name in ("pages", "out", "to", "map"):
                d[name].fill_(-9)

    torch.cuda.synchronize()
    for _ in range(10):
        for d in work:
            step(d)
    check()
    graphs = [torch.cuda.CUDAGraph() for _ in work]
    for d, g in zip(work, graphs):
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=d["stream"]):
            step(d)
    torch.cuda.synchronize()
    for _ in range(10):
        for d, g in zip(work, graphs):
            with torch.cuda.stream(d["stream"]):
                g.replay()
    check()
    assert pka.pka_get_device_error() == 0


def test_captured_large_fork_and_compact_replay():
    """The forms of several launches (tables past 65,536 entries, a pool past
    262,144 pages), captured and replayed back to back on other inputs."""
    rng = np.random.default_rng(12)
    pool = 300_000
    lens = rng.integers(2000, 4000, 20)
    indptr, ids, last = _parents(rng, lens, 1, pool)
    parent = rng.integers(0, 20, 50).astype(np.int32)
    pages = lens[parent] + 1
    child = np.concatenate([[0], np.cumsum(pages)]).astype(np.int32)
    r, idx = i32(np.zeros(pool)), i32(ids)
    table = torch.empty(int(child[-1]), dtype=torch.int32, device="cuda")
    src, dst, slots = (torch.empty(50, dtype=torch.int32, device="cuda") for _ in range(3))
    counts = torch.empty(2, dtype=torch.int32, device="cuda")
    held, r2, page_map = torch.empty_like(r), torch.empty_like(r), torch.empty_like(r)
    table2 = torch.empty_like(table)
    cs, cd = (torch.empty(pool // 2, dtype=torch.int32, device="cuda") for _ in range(2))
    ccounts = torch.empty(2, dtype=torch.int32, device="cuda")
    fixed = [i32(a) for a in (indptr, last, parent, child)]
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        pka.pka_fork_pages(1, r, fixed[0], idx, fixed[1], fixed[2], fixed[3], table, src, dst,
                           slots, counts, stream=stream)
        pka.pka_compact_pages(r, table, r2, table2, page_map, cs, cd, ccounts, stream=stream)
        held.copy_(r)
        pka.pka_free_pages(r, table, stream=stream)
    for seed in (1, 2, 3):
        rng = np.random.default_rng(seed)
        ids = rng.permutation(pool)[:len(ids)].astype(np.int32)
        refs = np.zeros(pool, np.int32)
        refs[ids] = 1
        r.copy_(i32(refs))
        idx.copy_(i32(ids))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        tables = [ids[indptr[i]:indptr[i + 1]].tolist() for i in range(20)]
        want, copies, after = cache.fork_pages(refs, tables, lens, 1, parent, pages)
        flat = np.concatenate(want)
        assert np.array_equal(_host(table), flat) and not copies
        assert np.array_equal(_host(held), after) and np.array_equal(_host(r), refs)
        w_refs, w_table, w_map, moves, live = cache.compact_pages(after, flat)
        assert np.array_equal(_host(r2), w_refs) and np.array_equal(_host(table2), w_table)
        assert np.array_equal(_host(page_map), w_map)
        assert _host(ccounts).tolist() == [len(moves), live]
        got = np.stack(_host(cs, cd), 1)[:len(moves)]
        assert np.array_equal(got, np.array(moves, np.int32))
    assert pka.pka_get_device_error() == 0


def test_captured_fork_and_return_replays():
    """Fork, copy and return captured (their first calls of this process may
    be these) and replayed with other tables and another pool content."""
    rng = np.random.default_rng(11)
    page, hk, d, pool = 4, 2, 64, 64
    params = pka.make_params(hk, hk, d, page)
    lens = np.array([14, 7, 9])
    indptr, ids, last = _parents(rng, lens, page, pool)
    parent, pages = np.array([2, 0, 0, 1], np.int32), np.array([4, 4, 5, 2])
    child = np.concatenate([[0], np.cumsum(pages)]).astype(np.int32)
    r, idx = i32(np.zeros(pool)), i32(ids)
    t = torch.zeros(2, pool, 2, page, hk, d, dtype=torch.bfloat16, device="cuda")
    table = torch.empty(int(child[-1]), dtype=torch.int32, device="cuda")
    src, dst, slots = (torch.empty(4, dtype=torch.int32, device="cuda") for _ in range(3))
    counts, held = torch.empty(2, dtype=torch.int32, device="cuda"), torch.empty_like(r)
    fixed = [i32(a) for a in (indptr, last, parent, child)]
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        pka.pka_fork_pages(page, r, fixed[0], idx, fixed[1], fixed[2], fixed[3], table, src, dst,
                           slots, counts, stream=stream)
        pka.pka_copy_pages(params, t[:, :, 0], t[:, :, 1], src, dst, slots, counts, stream=stream)
        held.copy_(r)
        pka.pka_free_pages(r, table, stream=stream)
    for seed in (1, 2, 3):
        rng = np.random.default_rng(seed)
        ids = rng.permutation(pool)[:len(ids)].astype(np.int32)
        refs = np.zeros(pool, np.int32)
        refs[ids] = 1
        x = _pool(rng, "bf16", tuple(t.shape))
        for a, b in ((r, i32(refs)), (idx, i32(ids)), (t, bf16(x))):
            a.copy_(b)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        tables = [ids[indptr[i]:indptr[i + 1]].tolist() for i in range(3)]
        want, copies, after = cache.fork_pages(refs, tables, lens, page, parent, pages)
        assert np.array_equal(_host(table), np.concatenate(want))
        assert np.array_equal(_host(held), after) and np.array_equal(_host(r), refs)
        s, e, n = (np.array(c) for c in zip(*copies))
        got = bits_of(t)
        for w in range(2):
            assert np.array_equal(got[:, :, w], cache.copy_pages(x[:, :, w], s, e, n))
    assert pka.pka_get_device_error() == 0


def test_large_takes_beside_small_ones_on_one_stream():
    """Two host threads share a stream and a pool: one takes and returns by the
    form of two launches, the other a few pages at a time.  A call's launches
    follow one another, so every take is whole and every page comes back."""
    rng = np.random.default_rng(17)
    refs = _refs(rng, 400_000, 40_000)
    r, stream, rounds = i32(refs), torch.cuda.Stream(), 400
    large = torch.full((rounds, 70_000), -9, dtype=torch.int32, device="cuda")
    small = torch.full((20_000, 64), -9, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    start, over, taken, errors = threading.Barrier(2), threading.Event(), [0], []

    def take(rows, until):
        try:
            start.wait(timeout=60)
            for pages in rows:
                pka.pka_alloc_pages(r, pages, stream=stream)
                pka.pka_free_pages(r, pages, stream=stream)
                if until is None:
                    taken[0] += 1
                    if over.is_set():
                        return
        except Exception as e:  # shown by the test's own thread
            errors.append(e)
        finally:
            if until is not None:
                until.set()

    threads = [threading.Thread(target=take, args=a) for a in ((list(large), over),
                                                               (list(small), None))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    got, few = _host(large, small[:taken[0]])
    free = refs == 0
    for pages in (got, few):
        assert pages.min() >= 0 and np.all(np.diff(pages, axis=1) > 0) and free[pages].all()
    assert np.array_equal(_host(r), refs)
    assert pka.pka_get_device_error() == 0


@pytest.mark.parametrize("pool", [200, 20_000])  # one block and a cluster
@pytest.mark.parametrize("page,where", [(4, 0), (4, 9), (4, -1), (1, 17)])
def test_fork_refuses_a_parent_page_that_nobody_holds(pool, page, where):
    """A shared page, or the partly filled one that would be copied, without a
    reference: nothing is written, whether or not the page would be taken."""
    rng = np.random.default_rng(pool + page)
    lens = np.array([38, 21])
    indptr, ids, last = _parents(rng, lens, page, pool)
    refs = np.zeros(pool, np.int32)
    refs[ids] = 1
    parent = np.array([1, 0, 0, -1], np.int32)
    pages = (indptr[1:] - indptr[:-1])[parent] + np.array([1, 0, 2, 0])
    _check_fork(page, refs, lens, indptr, ids, last, parent, pages)
    gap = ids[indptr[1] + where] if where < 0 else ids[where]
    refs[gap] = 0
    _, got = _fork(page, refs, indptr, ids, last, parent, pages)
    _refused(got, refs, METADATA)
    # a parent that no child continues may name what it will
    child = np.where(parent == 0, 1, parent)
    pages = (indptr[1:] - indptr[:-1])[1] + np.array([1, 0, 2, 0])
    _check_fork(page, refs, lens, indptr, ids, last, child, pages)


@pytest.mark.parametrize("what", ["parent_high", "parent_low", "short", "decreasing", "past_end",
                                  "last_zero", "last_high", "indptr", "indptr_past", "pages"])
def test_large_fork_refused(what):
    """The form of two launches: the second reads tables that the first has not
    checked yet, and neither writes anything."""
    rng = np.random.default_rng(19)
    lens = np.array([9001, 5005, 12000])
    indptr, ids, last = _parents(rng, lens, 4, 20_000)
    refs = np.zeros(20_000, np.int32)
    refs[ids] = 1
    parent, pages = np.array([0, 1, 2, 0, -1], np.int32), np.array([2251, 1253, 3001, 2252, 2])
    status = METADATA
    if what == "parent_high":
        parent[2] = 3
    if what == "parent_low":
        parent[2] = -2
    if what == "short":
        pages[3] = 2250
    if what == "decreasing":
        pages[4] = -1
    if what == "last_zero":
        last[1] = 0
    if what == "last_high":
        last[1] = 5
    if what == "indptr":
        indptr[1], indptr[2] = indptr[2], indptr[1]
    if what == "indptr_past":
        indptr[3] = 99_999
    if what == "pages":  # one free page too few
        refs[np.flatnonzero(refs == 0)[7:]] = 1
        status = WORKSPACE
    _, got = _fork(4, refs, indptr, ids, last, parent, pages, room=-1 if what == "past_end" else 9)
    _refused(got, refs, status)


def test_large_fork_takes_the_last_free_page():
    rng = np.random.default_rng(20)
    lens = np.array([9001, 5005, 12000])
    indptr, ids, last = _parents(rng, lens, 4, 20_000)
    refs = np.zeros(20_000, np.int32)
    refs[ids] = 1
    refs[np.flatnonzero(refs == 0)[8:]] = 1
    parent, pages = np.array([0, 1, 2, 0, -1], np.int32), np.array([2251, 1253, 3001, 2252, 2])
    _check_fork(4, refs, lens, indptr, ids, last, parent, pages)


@pytest.mark.parametrize("free", [0, 69_999, 70_000])
def test_large_take_with_too_few_free_takes_none(free):
    """The form of two launches: refused one page short, whole with the last."""
    rng = np.random.default_rng(free)
    refs = _refs(rng, 400_000, 400_000 - free)
    d, pages = i32(refs), torch.full((70_000,), 5, dtype=torch.int32, device="cuda")
    pka.pka_alloc_pages(d, pages)
    if free == 70_000:
        assert np.array_equal(_host(pages), np.flatnonzero(refs == 0))
        assert np.array_equal(_host(d), np.maximum(refs, 1))
        assert pka.pka_get_device_error() == 0
    else:
        assert np.all(_host(pages) == -1) and np.array_equal(_host(d), refs)
        assert pka.pka_get_device_error() == WORKSPACE
