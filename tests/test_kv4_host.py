"""K/V held in 4 bits without a GPU: the rounding rules pinned to worked groups
and closed forms, the page format, plans over such pools, and what the entry
points refuse before any device work.
"""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_attention_plan_gb300 as pka
from oracle import kv4
from paged_kv_attention_plan_gb300 import _pka
from tests.plan_image import parse

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 3, 4
A = 1 << 20  # an aligned address that a refused call never touches
INT4 = ["int4_g32", "int4_g64", "int4_g128"]


# ---------------------------------------------------------------------------
# The reference's rounding, on groups worked by hand
# ---------------------------------------------------------------------------

def test_worked_group():
    """0, 1, .., 15 twice: step 1, origin 0, every code its value."""
    code, step, origin = kv4.quantize(np.tile(np.arange(16.0), 2), 32)
    assert step[0] == 1 and origin[0] == 0
    assert np.array_equal(code, np.tile(np.arange(16), 2))
    assert np.array_equal(kv4.dequantize(code, step, origin), np.tile(np.arange(16.0), 2))


def test_ties_go_to_the_even_code():
    x = np.zeros(32)
    x[:4] = [0.5, 1.5, 2.5, 14.5]
    x[31] = 15
    code, step, _ = kv4.quantize(x, 32)
    assert step[0] == 1 and list(code[:4]) == [0, 2, 2, 14]


def test_error_is_half_a_step_and_the_words_roundings():
    """|x - value| <= step / 2 inside the codes' reach; at its ends the bf16 step
    may reach short by 15 half-steps of 2^-8 and the origin's rounding comes on top."""
    rng = np.random.default_rng(0)
    for g in (32, 64, 128):
        x = rng.standard_normal((200, 128)).astype(np.float32) * 10 + 3
        code, step, origin = kv4.quantize(x, g)
        err = np.abs(kv4.dequantize(code, step, origin) - x).reshape(200, -1, g)
        lo = np.abs(x.reshape(200, -1, g).min(-1))
        tol = step * (0.5 + 15 * 2.0 ** -8) + lo * 2.0 ** -8 + 2.0 ** -20
        assert np.all(err <= tol[..., None])


def test_groups_without_a_range_and_not_finite():
    same = np.full(32, -3.25, np.float32)
    code, step, origin = kv4.quantize(same, 32)
    assert step[0] == 0 and origin[0] == -3.25 and not code.any()
    for bad in (np.nan, np.inf, -np.inf):
        x = np.arange(32, dtype=np.float32)
        x[5] = bad
        assert np.isnan(kv4.dequantize(*kv4.quantize(x, 32))).all()
    tiny = np.zeros(32, np.float32)
    tiny[3] = np.float32(2.0 ** -130)
    assert kv4.quantize(tiny, 32)[1][0] == 0


@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("dim,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)])
def test_pool_round_trip(layout, dim, group):
    """A slot written reads back as its quantised rows, and no other byte changes."""
    rng = np.random.default_rng(dim + group)
    pool = kv4.Pool.empty(3, 5, 3, dim, group, layout, fill=0xAB)
    x = rng.standard_normal((3, dim)).astype(np.float32)
    before = pool.data.copy()
    pool.write(1, 4, x)
    want = kv4.dequantize(*kv4.quantize(x, group))
    assert np.array_equal(pool.read(1, 4), want)
    assert (pool.data != before).sum() <= 3 * (dim // 2 + 4 * dim // group)
    assert np.array_equal(pool.data[[0, 2]], before[[0, 2]])


def test_reference_attention_against_softmax():
    """The reference equals the plain attention reference on the pools' values,
    where these are bf16 numbers (steps of 1/2, origins of multiples of 1/2)."""
    from oracle import ref
    from inputs import workloads as W
    rng = np.random.default_rng(1)
    b = W.make_paged_batch(3, [3, 1, 4], [6, 2, 9], page_size=4, hq=4, hk=2, d=64)
    kp, vp = (kv4.Pool.empty(b.k_pool.shape[0], 4, 2, 64, 32, "NHD") for _ in range(2))
    for p in (kp, vp):
        x = [rng.integers(0, 16, (int(n), 2, 64)) / 2 - 4 for n in b.kv_lens]
        for rows in x:
            rows[..., 0::32], rows[..., 1::32] = -4, 3.5  # a range of 15 half steps
        kv4.fill(p, b.kv_indptr, b.kv_indices, b.kv_lens, x)
    kw = dict(qo_indptr=b.qo_indptr, kv_indptr=b.kv_indptr, kv_indices=b.kv_indices)
    vals = []
    for p in (kp, vp):
        x = np.stack([[p.read(i, s) for s in range(4)] for i in range(p.data.shape[0])])
        vals.append((x.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16))
        assert np.array_equal(ref.bf16_bits_to_f64(vals[-1]), x)
    want = ref.batch_attention(b.q, *vals, last_page_len=b.last_page_len, page_size=4,
                               num_qo_heads=4, num_kv_heads=2, **kw)
    got = kv4.attention(b.q, kp, vp, kv_lens=b.kv_lens, hq=4, hk=2, **kw)
    for x, y in zip(got, want):
        assert np.abs(x - y).max() < 1e-12


# ---------------------------------------------------------------------------
# The library on the host
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("kv", INT4)
@pytest.mark.parametrize("heads,page", [(1, 1), (2, 16), (7, 3), (8, 64)])
def test_page_bytes(dim, kv, heads, page):
    p = pka.make_params(heads, heads, dim, page, kv_dtype=kv)
    group = int(kv[6:])
    if group > dim:
        with pytest.raises(pka.PkaError) as e:
            pka.pka_kv_page_bytes(p)
        assert e.value.status == UNSUPPORTED
    else:
        assert pka.pka_kv_page_bytes(p) == kv4.page_bytes(page, heads, dim, group)
        assert _pka._page_bytes(p) == kv4.page_bytes(page, heads, dim, group)


def test_page_bytes_of_other_types_and_refusals():
    assert pka.pka_kv_page_bytes(pka.make_params(4, 2, 64, 16)) == 16 * 2 * 64 * 2
    assert pka.pka_kv_page_bytes(pka.make_params(4, 2, 64, 16, kv_dtype="e4m3")) == 16 * 2 * 64
    n = ctypes.c_int64()
    L = _pka.lib()

    def call(p, out=n):
        return L.pka_kv_page_bytes(ctypes.byref(p) if p else None,
                                   ctypes.byref(out) if out is not None else None)
    good = pka.make_params(4, 2, 64, 16)
    assert call(None) == INVALID and call(good, None) == INVALID
    assert call(pka.make_params(4, 2, 96, 16)) == UNSUPPORTED
    assert call(pka.make_params(4, 2, 64, 16, kv_ragged=True)) == UNSUPPORTED
    bad = pka.make_params(4, 2, 64, 16)
    bad.kv_dtype = 5
    assert call(bad) == INVALID
    # pages of 2 GB and more
    assert call(pka.make_params(8, 8, 128, 1 << 22, kv_dtype="int4_g128")) == UNSUPPORTED


def _i32(*x):
    return np.array(x, np.int32)


@pytest.mark.parametrize("kv", INT4)
def test_validate(kv):
    batch = (_i32(0, 1, 2), _i32(0, 1, 3), _i32(2, 4))
    assert pka.pka_validate(pka.make_params(8, 2, 128, 4, kv_dtype=kv), *batch) == OK
    assert pka.pka_validate(pka.make_params(8, 2, 128, 4, kv_dtype=kv, kv_ragged=True),
                            *batch) == UNSUPPORTED
    want = UNSUPPORTED if kv == "int4_g128" else OK
    assert pka.pka_validate(pka.make_params(8, 2, 64, 4, kv_dtype=kv), *batch) == want


def _plan(params, qo, kv, last):
    h = pka.pka_plan_create()
    try:
        buf = np.zeros(1 << 20, np.uint8)
        s = pka.pka_plan(h, params, qo, kv, last, None, buf, check=False)
        return s, pka.pka_plan_get_info(h), parse(buf) if s == OK else None
    finally:
        pka.pka_plan_destroy(h)


@pytest.mark.parametrize("kv", INT4)
def test_plans_decode_rows_apart_and_others_over_a_scratch(kv):
    """The plan is that of e4m3 pools: the same items, and the keys of the rows
    with qo_len >= 2 decoded to the scratch."""
    qo, ptr, last = _i32(0, 1, 4, 5, 5), _i32(0, 3, 5, 6, 7), _i32(2, 4, 1, 3)
    got, want = (_plan(pka.make_params(8, 2, 128, 4, kv_dtype=t, num_sms=152), qo, ptr, last)
                 for t in (kv, "e4m3"))
    assert got[0] == want[0] == OK
    a, b = got[1].as_dict(), want[1].as_dict()
    # beside the keys: 5 rows of Q in f16, their scales, and a word a kv head and pool
    staged = 5 * 8 * 128 * 2 + 256 + 256
    assert a.pop("float_ws_bytes") == b.pop("float_ws_bytes") + staged
    # a decode CTA's share counts what its items cost besides their keys
    assert a.pop("decode_chunk_tokens") >= b.pop("decode_chunk_tokens")
    for x in (a, b):
        for k in ("num_decode_ctas", "int_ws_bytes"):
            x.pop(k)
    assert a == b and a["kv_scratch_rows"] == 8
    for k in ("prefill_items", "merges", "joins"):
        assert got[2][k] == want[2][k]


@pytest.mark.parametrize("seed", range(12))
def test_decode_plans_fill_the_sms_once(seed):
    """Over 4-bit pools no plan has more decode CTAs than SMs, whatever the lengths,
    every key is covered once, and CTAs of many short requests close early."""
    from inputs import workloads as W
    from tests.test_host_abi import check_coverage
    rng = np.random.default_rng(seed)
    n = int(rng.integers(1, 400))
    kv = rng.integers(1, [2, 40, 3000, 20000][seed % 4], n)
    hq, hk = [(32, 8), (8, 1), (28, 7), (64, 16)][seed // 3]
    b = W.make_paged_batch(seed, np.ones(n, np.int32), kv, page_size=16, hq=hq, hk=hk, d=128,
                           is_decode=True, with_payload=False)
    p = pka.make_params(hq, hk, 128, 16, kv_dtype="int4_g64", num_sms=152)
    s, info, plan = _plan(p, b.qo_indptr, b.kv_indptr, b.last_page_len)
    assert s == OK and info.num_decode_ctas <= 152
    check_coverage(plan, b, hq, hk, True, info)
    ptr = plan["decode_cta_ptr"]
    per = [ptr[i + 1] - ptr[i] for i in range(len(ptr) - 1)]
    if seed % 4 == 0:  # single keys: dealt evenly
        assert max(per) <= -(-len(plan["decode_items"]) // 152) + 1


@pytest.mark.parametrize("seed", range(24))
def test_decode_shares_are_found_in_few_tries(seed):
    """The share of a CTA is tried in steps of an eighth of an item's cost from its least value
    on; it never goes past that value by two items' cost, two tiles and a step."""
    rng = np.random.default_rng(100 + seed)
    n, sms = int(rng.integers(1, 1500)), int(rng.choice([1, 7, 148, 152]))
    kv = rng.integers(1, [2, 17, 300, 9000][seed % 4], n)
    hq, hk = [(32, 8), (8, 1), (13, 13), (64, 16)][seed // 6]
    ptr = np.concatenate([[0], np.cumsum(kv)]).astype(np.int32)
    p = pka.make_params(hq, hk, 128, 1, kv_dtype="int4_g64", num_sms=sms)
    h = pka.pka_plan_create()
    buf = np.zeros(16 << 20, np.uint8)
    s = pka.pka_plan(h, p, None, ptr, np.ones(n, np.int32), None, buf, check=False)
    assert s == OK
    info = pka.pka_plan_get_info(h)
    per_cta = parse(buf)["header"]["decode_heads_per_cta"]
    pka.pka_plan_destroy(h)
    units = hk // per_cta
    over = 896 // per_cta  # keys that an item costs besides its own
    least = max(-(-int(kv.sum() * units + over * n * units) // sms), 64 + over)
    assert info.num_decode_ctas <= sms
    assert info.decode_chunk_tokens <= least + 2 * over + 32 + (over // 8 + 15) // 16 * 16


@pytest.mark.parametrize("lens", [(1, 33, 0, 250), (0,), (0, 0, 5000, 0), (64, 0, 64)])
def test_rows_without_keys_are_planned(lens):
    """A decode row whose request has no keys is an item of none, which writes its zeros;
    ragged K/V, where lengths of 0 are allowed."""
    n = len(lens)
    p = pka.make_params(16, 4, 128, 1, mask_mode="none", kv_ragged=True, num_sms=152)
    kv = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    s, info, plan = _plan(p, np.arange(n + 1, dtype=np.int32), kv, None)
    assert s == OK
    keys = {r: 0 for r in range(n)}
    for w in plan["decode_items"]:
        keys[w["q_row0"]] += w["t1"] - w["t0"]
    assert {w["q_row0"] for w in plan["decode_items"]} == set(range(n))
    assert [keys[r] for r in range(n)] == list(lens)
    assert plan["decode_cta_ptr"][-1] == len(plan["decode_items"])


@pytest.mark.parametrize("kv", INT4)
def test_paged_requests_without_pages(kv):
    """Paged requests hold at least one key: refused, as for bf16 pools."""
    qo, ptr, last = _i32(0, 1, 2, 3), _i32(0, 2, 2, 5), _i32(4, 0, 1)
    for t in (kv, "bf16"):
        assert _plan(pka.make_params(8, 2, 128, 4, kv_dtype=t, num_sms=152), qo, ptr,
                     last)[0] not in (OK, UNSUPPORTED)


@pytest.mark.parametrize("kv", INT4 + ["e4m3"])
def test_items_over_a_scratch_name_their_unit(kv):
    """An item of the tensor cores knows whose keys it reads: 4-bit pools keep the scales
    of the staged rows by request and kv head, so that requests share none."""
    n = 60
    qo = np.concatenate([[0], np.cumsum(1 + np.arange(n) % 3)]).astype(np.int32)
    ptr = np.concatenate([[0], np.cumsum(1 + np.arange(n) % 5)]).astype(np.int32)
    last = np.full(n, 4, np.int32)
    s, info, plan = _plan(pka.make_params(8, 2, 128, 4, kv_dtype=kv, num_sms=152), qo, ptr, last)
    assert s == OK
    units = plan["dequant_units"]
    assert len(units) == 40 and len({w["join"] for w in plan["prefill_items"]}) == 40
    for w in plan["prefill_items"]:
        u = units[w["join"]]
        assert u["dst_row0"] == w["kv_base"] and u["kv_base"] == ptr[w["req"]]
        assert u["kv_len"] == w["kv_len"]
    if kv != "e4m3":  # beside e4m3's: staged Q, its scales, and two bounds a unit and kv head
        want = _plan(pka.make_params(8, 2, 128, 4, kv_dtype="e4m3", num_sms=152), qo, ptr, last)
        rows = int(qo[-1])
        more = rows * 8 * 128 * 2 + rows * 8 * 4 + 40 * 2 * 8
        assert info.float_ws_bytes >= want[1].float_ws_bytes + more


@pytest.mark.parametrize("kv", INT4)
def test_graph_mode_needs_the_scratch_capacity(kv):
    kw = dict(kv_dtype=kv, graph_max_batch=4, graph_max_qo_rows=16, num_sms=152)
    ptr, last = _i32(0, 3, 5), _i32(2, 4)
    decode, mixed = _i32(0, 1, 2), _i32(0, 1, 4)
    assert _plan(pka.make_params(8, 2, 128, 4, **kw), decode, ptr, last)[0] == OK
    assert _plan(pka.make_params(8, 2, 128, 4, **kw), mixed, ptr, last)[0] == UNSUPPORTED
    kw["graph_max_kv_tokens"] = 8
    assert _plan(pka.make_params(8, 2, 128, 4, **kw), mixed, ptr, last)[0] == OK
    kw["graph_max_kv_tokens"] = 7
    assert _plan(pka.make_params(8, 2, 128, 4, **kw), mixed, ptr, last)[0] == WORKSPACE


# ---------------------------------------------------------------------------
# Refusals (raw C calls: every pointer is a number that is never read)
# ---------------------------------------------------------------------------

def _append(p, stride=None, k_new=A, v_new=A, app=A, ptr=A, idx=A, last=A, k=A, v=A, nnz=3,
            batch=2):
    stride = kv4.page_bytes(4, 2, 128, 128) if stride is None else stride
    return _pka.lib().pka_append_paged_kv_cache(ctypes.byref(p), batch, k_new, v_new, app, nnz,
                                                ptr, idx, last, k, v, stride, None)


@pytest.fixture
def p4():
    return pka.make_params(8, 2, 128, 4, kv_dtype="int4_g128")


@pytest.mark.parametrize("kw", [
    dict(k_new=None), dict(v_new=None), dict(app=None), dict(ptr=None), dict(idx=None),
    dict(last=None), dict(k=None), dict(v=None), dict(k_new=A + 8), dict(v=A + 8), dict(app=A + 2),
    dict(idx=A + 1), dict(stride=0), dict(stride=-544), dict(stride=544 + 8), dict(stride=528),
    dict(nnz=-1), dict(batch=-1)])
def test_append_refusals(p4, kw):
    assert _append(p4, **kw) == INVALID


def test_append_unsupported(p4):
    assert _append(p4, nnz=(1 << 33) + 1) == UNSUPPORTED
    assert _append(pka.make_params(8, 2, 64, 4, kv_dtype="int4_g128")) == UNSUPPORTED
    assert _append(pka.make_params(5000, 5000, 128, 4, kv_dtype="int4_g128")) == UNSUPPORTED
    assert _append(p4, nnz=0, k=None) == OK and _append(p4, batch=0, k=None) == OK


def _read(p, begin=A, ind=A, ptr=A, idx=A, last=A, k=A, v=A, stride=None, pages=9, ko=A, vo=A,
          nnz=3, batch=2):
    stride = 544 if stride is None else stride
    return _pka.lib().pka_read_paged_kv_cache(ctypes.byref(p), batch, begin, ind, nnz, ptr, idx,
                                              last, k, v, stride, pages, ko, vo, None)


@pytest.mark.parametrize("kw", [
    dict(ind=None), dict(ptr=None), dict(idx=None), dict(last=None), dict(k=None), dict(v=None),
    dict(begin=A + 2), dict(ind=A + 1), dict(idx=A + 2), dict(k=A + 4), dict(v=A + 8),
    dict(ko=A + 8), dict(vo=A + 4), dict(stride=0), dict(stride=552), dict(stride=528),
    dict(nnz=-1), dict(batch=-1), dict(pages=-1)])
def test_read_refusals(p4, kw):
    assert _read(p4, **kw) == INVALID


def test_read_unsupported_and_nothing_to_do(p4):
    assert _read(p4, nnz=(1 << 33) + 1) == UNSUPPORTED
    assert _read(pka.make_params(8, 2, 64, 4, kv_dtype="int4_g128")) == UNSUPPORTED
    assert _read(pka.make_params(8, 2, 96, 4)) == UNSUPPORTED
    assert _read(pka.make_params(8, 2, 64, 4, kv_ragged=True)) == UNSUPPORTED
    assert _read(pka.make_params(5000, 5000, 128, 4)) == UNSUPPORTED
    for kw in (dict(nnz=0), dict(batch=0), dict(ko=None, vo=None)):
        assert _read(p4, k=None, **kw) == OK
    # a stride in elements: bf16 pools take whole 8, e4m3 whole 16
    assert _read(pka.make_params(8, 2, 64, 4), stride=4 * 2 * 64 + 4) == INVALID
    assert _read(pka.make_params(8, 2, 64, 4, kv_dtype="e4m3"), stride=4 * 2 * 64 + 8) == INVALID


def test_rope_append_and_copy_refuse_short_strides_and_wide_groups(p4):
    rope = pka.make_rope(128)

    def append(p, stride):
        return _pka.lib().pka_rope_append_paged_kv_cache(
            ctypes.byref(p), ctypes.byref(rope), 2, 3, None, 0, None, A, 256, A, 256, None, A, A,
            A, A, A, A, stride, 9, None)

    def copy(p, stride):
        return _pka.lib().pka_copy_pages(ctypes.byref(p), 1, A, A, stride, 0, 9, A, A, None, 3,
                                         None, None)
    for f in (append, copy):
        assert f(p4, 528) == INVALID and f(p4, 552) == INVALID
        assert f(pka.make_params(8, 2, 64, 4, kv_dtype="int4_g128"), 544) == UNSUPPORTED
        assert f(pka.make_params(8, 2, 128, 4, kv_dtype="int4_g128", kv_ragged=True),
                 544) == UNSUPPORTED


def test_binding_refuses_tensors_off_the_device(p4):
    cpu = torch.zeros(3, 544, dtype=torch.uint8)
    with pytest.raises(TypeError):
        _pka._dev_pool(cpu, "k", p4)
    with pytest.raises(ValueError):
        _pka._int4_pages(torch.zeros(3, 528, dtype=torch.uint8), "k", p4)
    with pytest.raises(ValueError):
        _pka._int4_pages(torch.zeros(3, 1088, dtype=torch.uint8)[:, ::2], "k", p4)
    _pka._int4_pages(torch.zeros(3, 2, 544, dtype=torch.uint8)[:, 1], "k", p4)


def test_append_binding_refuses_rows_tables_and_strides_that_do_not_fit(monkeypatch):
    """Rows of K and V alike, tables of one batch, and the pools' own stride: the kernel
    reads V by K's row count and trusts the table.  (Checked on host tensors, with the
    library's entry replaced.)"""
    calls = []

    class Library:
        @staticmethod
        def pka_append_paged_kv_cache(*args):
            calls.append(args)
            return 0

    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)  # host tensors' device
    monkeypatch.setattr(_pka, "lib", lambda: Library)
    p = pka.make_params(8, 2, 128, 4, kv_dtype="int4_g128")
    pools = torch.zeros(5, 2, 544, dtype=torch.uint8)
    rows = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    table = [torch.tensor(x, dtype=torch.int32) for x in ([0, 1, 3], [0, 1, 2], [0, 1], [1, 2])]

    def append(k_new=rows, v_new=rows, table=table, k=pools[:, 0], v=pools[:, 1], stride=1088):
        return pka.pka_append_paged_kv_cache(p, k_new, v_new, *table, k, v, stride, stream=0)

    assert append() == 0 and append(k=pools[:1, 0], v=pools[:1, 1], stride=544) == 0
    assert len(calls) == 2
    longer = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    for kw in (dict(v_new=rows[:2]), dict(k_new=longer), dict(k_new=longer[:3, :1].contiguous()),
               dict(k_new=longer[..., :64].contiguous(), v_new=longer[..., :64].contiguous()),
               dict(k_new=rows.view(3, 256), v_new=rows.view(3, 256)),
               dict(table=[table[0], table[1][:2]] + table[2:]),
               dict(table=table[:3] + [table[3][:1]]),
               dict(stride=544), dict(stride=2176), dict(stride=0),
               dict(k=pools, v=pools, stride=1088), dict(k=pools, v=pools, stride=544),
               dict(v=pools[:, 1].contiguous())):
        with pytest.raises(ValueError):
            append(**kw)
    assert len(calls) == 2


def test_runs_refuse_pools_of_several_layers_and_strides_of_their_own(p4):
    """A run takes one layer's pages, K's and V's the same stride apart: a pool of all
    layers would be read a layer apart."""
    pools = torch.zeros(3, 5, 2, 544, dtype=torch.uint8)  # layers, pages, K and V
    for t in (pools, pools[:, :, 0], pools[0], pools[0, 0, 0]):
        with pytest.raises(ValueError):
            _pka._int4_pages(t, "k", p4)
    k, v = pools[0, :, 0], pools[0, :, 1]
    _pka._int4_pages(k, "k", p4)
    _pka._int4_strides(k, v, 1088)
    _pka._int4_strides(k[:1], v[:1], 544)  # one page: its stride leads nowhere
    for kk, vv, stride in ((k, v, 544), (k, v.contiguous(), 1088), (k.contiguous(), v, 544)):
        with pytest.raises(ValueError):
            _pka._int4_strides(kk, vv, stride)
