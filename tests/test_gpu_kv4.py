"""GPU parity of the operators over K/V held in 4 bits against the float64
reference: the appends (plain and rotating), the read-back, page copies, and
attention over the pools (decode rows, rows through the f16 scratch, cascades,
captured runs).

Tolerances.
Appends are exact, bytes and words: differences of bf16 values and products
with steps are exact or far from a tie, so the library's codes are the
reference's.  A rotating append starts from rotated float32 values off by up to
2^-20 m (|a| + |b|) (see test_gpu_rope.py); its values are compared with the
reference's of the float64 rotation: both err from the true value by half a
step and the words' roundings, so they differ by at most one step more than
the inputs do.

Decode rows, with A = the largest sum of magnitudes of a score (log2 units) and
V = the weighted sum of magnitudes |step| c + |origin| of an output.  A score
sums at most 128 products in MMAs of 16 and then a few terms, each rounding at
most 2^-23 of the magnitudes (accumulation may truncate): 2^-23 (128/16 + 8)
<= 2^-19 A.  A probability is ex2 of it, 2^-22, with m and l rounding alike, so
an output's weights are off by a relative r = 2 ln2 2^-19 A + 2^-20, on both
sides of the quotient.  P with V's step rounds to f16, half a step 2^-11; the
sums over up to 2^13 keys round 2^-23 a step of 16 keys each, 2^-14 at most,
and merges 2^-20.  So |o - o_ref| <= (2 r + 2^-11 + 2^-13) V + 2^-8 |o_ref|,
and the statistic is within 2^-19 A + 2^-19 (1 + |lse|).

Rows with qo_len >= 2 read K and V rounded to f16, half a step 2^-11 a value.
A score's 128 roundings are independent of one another and of the sign, so
their sum has a standard deviation of at most 2^-11 / sqrt(3) times the root of
the sum of squares of its products (A2), and six of these are 3.5 2^-11 A2,
which takes the place of the first term above: s = 3.5 2^-11 A2 + 2^-19 A,
r = 2 ln2 s + 2^-20.  V's own rounding adds 2^-11 V to P's.  Where a request's
groups of a kv head are more than 2^16 apart, its rows, P and V round to bf16,
half a step 2^-8: 2^-8 in the places of 2^-11.  P in f16 has 11 bits down to 2^-25 of
the largest probability; below, half its last step is 2^-25 where the largest is at
least 2^11: an output sums errors of 2^-36 of each |v| more.
"""
import numpy as np
import pytest
import torch

import paged_kv_attention_plan_gb300 as pka
from inputs import workloads as W
from oracle import cache, kv4, ref
from tests.gpu_util import bf16, bits_of, f64, i32

pytestmark = pytest.mark.gpu

SHAPES = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)]


def _name(group):
    return f"int4_g{group}"


def _dev(pool):
    return torch.from_numpy(pool.data.copy()).cuda()


class Batch:
    """A paged batch over 4-bit pools, every cached slot a quantised row and the
    others (free pages, slots behind a request's last) the bytes 0xFF: words of
    NaN and codes of 15."""

    def __init__(self, seed, kv_lens, *, qo_lens=None, page=4, layout="NHD", hq=8, hk=2, d=128,
                 group=128, spread=1.0):
        rng = np.random.default_rng(seed)
        self.kv_lens = np.asarray(kv_lens, np.int32)
        n = len(kv_lens)
        self.qo_lens = np.ones(n, np.int32) if qo_lens is None else np.asarray(qo_lens, np.int32)
        self.qo_indptr = np.concatenate([[0], np.cumsum(self.qo_lens)]).astype(np.int32)
        pages = int((-(-self.kv_lens // page)).sum()) + 3
        self.kv_indptr, self.kv_indices, self.last, _ = W.build_page_table(
            rng, self.kv_lens, page, pool_pages=pages)
        self.page, self.layout, self.hq, self.hk, self.d, self.group = page, layout, hq, hk, d, group
        self.q = W.normal_bf16_bits(rng, (int(self.qo_indptr[-1]), hq, d))
        self.k, self.v = (kv4.Pool.empty(pages, page, hk, d, group, layout, fill=0xFF)
                          for _ in range(2))
        for p in (self.k, self.v):
            kv4.fill(p, self.kv_indptr, self.kv_indices, self.kv_lens,
                     [spread * rng.standard_normal((int(m), hk, d)) for m in self.kv_lens])

    def params(self, **kw):
        return dict(num_qo_heads=self.hq, num_kv_heads=self.hk, head_dim=self.d,
                    page_size=self.page, layout=self.layout, kv_dtype=_name(self.group), **kw)

    def make_params(self):
        return pka.make_params(self.hq, self.hk, self.d, self.page, self.layout,
                               kv_dtype=_name(self.group))

    def table(self):
        return i32(self.kv_indptr), i32(self.kv_indices), i32(self.last)

    def run(self, attn=None, mask=None, stream=None, **kw):
        attn = attn or pka.BatchAttention()
        kw.setdefault("mask_mode", "causal")
        info = attn.plan(self.qo_indptr, self.kv_indptr, self.last, **self.params(**kw))
        o, lse = attn.run(bf16(self.q), _dev(self.k), _dev(self.v), i32(self.kv_indices), mask)
        torch.cuda.synchronize()
        assert pka.pka_get_device_error() == 0
        return f64(o), f64(lse), info

    def want(self, **kw):
        return kv4.attention(self.q, self.k, self.v, qo_indptr=self.qo_indptr,
                             kv_indptr=self.kv_indptr, kv_indices=self.kv_indices,
                             kv_lens=self.kv_lens, hq=self.hq, hk=self.hk, **kw)


def _assert_decode(o, lse, want, rows=None, staged=False):
    ow, lw, a_k, a_v, a_2 = want if rows is None else tuple(x[rows] for x in want)
    if rows is not None:
        o, lse = o[rows], lse[rows]
    score = 2.0 ** -19 * a_k + (3.5 * 2.0 ** -11 * a_2 if staged else 0)
    r = 2 * np.log(2) * score[..., None] + 2.0 ** -20
    tol = (2 * r + (2 if staged else 1) * 2.0 ** -11 + 2.0 ** -13) * a_v + 2.0 ** -8 * np.abs(ow)
    assert np.all(np.isfinite(o)) and np.all(np.abs(o - ow) <= tol)
    fin = np.isfinite(lw)
    assert np.array_equal(fin, np.isfinite(lse)) and np.all(lse[~fin] == -np.inf)
    lse, lw, score = lse[fin], lw[fin], score[fin]
    assert np.all(np.abs(lse - lw) <= score + 2.0 ** -19 * (1 + np.abs(lw)))


def _assert_staged(o, lse, want, rows=None):
    _assert_decode(o, lse, want, rows, staged=True)


def _assert_wide(o, lse, want, rows=None):
    rows = slice(None) if rows is None else rows
    o, lse, (ow, lw, a_k, a_v, a_2) = o[rows], lse[rows], (x[rows] for x in want)
    score = 2.0 ** -19 * a_k + 3.5 * 2.0 ** -8 * a_2
    r = 2 * np.log(2) * score[..., None] + 2.0 ** -20
    tol = (2 * r + 2 * 2.0 ** -8 + 2.0 ** -13) * a_v + 2.0 ** -8 * np.abs(ow)
    assert np.all(np.isfinite(o)) and np.all(np.abs(o - ow) <= tol)
    fin = np.isfinite(lw)
    assert np.array_equal(fin, np.isfinite(lse)) and np.all(lse[~fin] == -np.inf)
    lse, lw, score = lse[fin], lw[fin], score[fin]
    assert np.all(np.abs(lse - lw) <= score + 2.0 ** -19 * (1 + np.abs(lw)))


# ---------------------------------------------------------------------------
# Appends
# ---------------------------------------------------------------------------

def _append_case(seed, new, prefix, page, layout, hk, d, group, rows=None):
    rng = np.random.default_rng(seed)
    new, total = np.asarray(new), np.asarray(new) + np.asarray(prefix)
    pages = int((-(-total // page)).sum()) + 2
    ptr, idx, last, _ = W.build_page_table(rng, total, page, pool_pages=pages)
    app = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    n = int(app[-1])
    k, v = (W.normal_bf16_bits(rng, (n, hk, d)) if rows is None else rows for _ in range(2))
    pool = kv4.Pool.empty(pages, page, hk, d, group, layout, fill=0x5A)
    return k, v, app, ptr, idx, last, pool


def _appended(pool, x, app, ptr, idx, last):
    out = pool.copy()
    for row, _, page, slot in cache.append_slots(app, ptr, idx, last, pool.P):
        out.write(page, slot, x[row].astype(np.float32))
    return out.data


@pytest.mark.parametrize("d,group", SHAPES)
@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("new,prefix,page,hk", [
    ([1], [0], 1, 1), ([1, 1, 1], [0, 5, 16], 16, 8), ([3, 0, 18, 1], [1, 7, 0, 30], 4, 2),
    ([7, 2], [0, 3], 3, 5), ([40], [9], 16, 7)])
def test_append(d, group, layout, new, prefix, page, hk):
    k, v, app, ptr, idx, last, pool = _append_case(d + hk, new, prefix, page, layout, hk, d, group)
    kp, vp = _dev(pool), _dev(pool)
    params = pka.make_params(hk, hk, d, page, layout, kv_dtype=_name(group))
    pka.pka_append_paged_kv_cache(params, bf16(k), bf16(v), i32(app), i32(ptr), i32(idx),
                                  i32(last), kp, vp, kp.stride(0))
    torch.cuda.synchronize()
    for x, p in ((k, kp), (v, vp)):
        want = _appended(pool, ref.bf16_bits_to_f64(x), app, ptr, idx, last)
        assert np.array_equal(p.cpu().numpy(), want)
    assert pka.pka_get_device_error() == 0


@pytest.mark.parametrize("d,group", SHAPES)
def test_append_of_odd_groups(d, group):
    """Groups of one value, zeros of both signs, ties, ranges beyond bf16's middle,
    of the smallest numbers, and groups with NaN or an infinity."""
    rows = np.zeros((12, 2, d), np.float32)
    g = np.arange(d) % group
    rows[0] = -3.25
    rows[1] = np.where(g % 2, 0.0, -0.0)
    rows[2] = np.where(g < 16, np.minimum(g, 15), 7.5)       # a step of 1 and its tie
    rows[3] = np.where(g == 1, 3.0e38, -1.0)
    rows[4] = np.where(g == 1, 3.0e38, np.where(g == 2, -3.0e38, 0.0))  # range past float32
    rows[5] = np.where(g == 3, 2.0 ** -130, 0.0)
    rows[6] = np.where(g == 3, 2.0 ** -121, 2.0 ** -122)
    rows[7] = np.where(g == 5, np.nan, 1.0)
    rows[8] = np.where(g == group - 1, np.inf, 1.0)
    rows[9] = np.where(g == 0, -np.inf, g)
    rows[10, 0] = np.where(np.arange(d) == 0, np.nan, 1.0)   # NaN in one group alone
    rows[10, 1] = 2.5 - g
    rows[11] = 1000.0 + g * 8.0
    bits = kv4.bf16_round(rows).view(np.uint32) >> 16
    bits = np.where(np.isnan(rows), 0x7FC0, bits).astype(np.uint16)
    k, v, app, ptr, idx, last, pool = _append_case(1, [12], [3], 4, "NHD", 2, d, group, bits)
    kp, vp = _dev(pool), _dev(pool)
    params = pka.make_params(2, 2, d, 4, kv_dtype=_name(group))
    pka.pka_append_paged_kv_cache(params, bf16(k), bf16(v), i32(app), i32(ptr), i32(idx),
                                  i32(last), kp, vp, kp.stride(0))
    torch.cuda.synchronize()
    want = _appended(pool, ref.bf16_bits_to_f64(bits), app, ptr, idx, last)
    # -0 or +0 may be the least of a group of both: compare values there
    got = pool.copy()
    got.data[:] = kp.cpu().numpy()
    exp = pool.copy()
    exp.data[:] = want
    for row, _, page, slot in cache.append_slots(app, ptr, idx, last, 4):
        assert np.array_equal(got.read(page, slot), exp.read(page, slot), equal_nan=True), row
    assert np.isnan(got.read(*cache.append_slots(app, ptr, idx, last, 4)[7][2:])).any()


def test_append_leaves_padded_rows_and_bad_positions():
    """Rows behind the last request are left out; a row whose position lies before
    its request's first slot is not appended and the violation is noted."""
    k, v, app, ptr, idx, last, pool = _append_case(5, [2, 3], [1, 4], 4, "HND", 2, 128, 64)
    params = pka.make_params(2, 2, 128, 4, "HND", kv_dtype="int4_g64")
    pad = np.concatenate([k, np.full((4, 2, 128), 0x4040, np.uint16)])
    kp, vp = _dev(pool), _dev(pool)
    pka.pka_append_paged_kv_cache(params, bf16(pad), bf16(pad), i32(app), i32(ptr), i32(idx),
                                  i32(last), kp, vp, kp.stride(0))
    torch.cuda.synchronize()
    want = _appended(pool, ref.bf16_bits_to_f64(k), app, ptr, idx, last)
    assert np.array_equal(kp.cpu().numpy(), want) and pka.pka_get_device_error() == 0
    # request 0 holds 3 slots: of 5 appended rows the first two have none
    far = np.array([0, 5, 5], np.int32)
    kp, vp = _dev(pool), _dev(pool)
    pka.pka_append_paged_kv_cache(params, bf16(k), bf16(k), i32(far), i32(ptr), i32(idx),
                                  i32(last), kp, vp, kp.stride(0))
    torch.cuda.synchronize()
    assert pka.pka_get_device_error() == 2
    out = pool.copy()
    for j in range(3):
        out.write(int(idx[ptr[0]]), j, ref.bf16_bits_to_f64(k[2 + j]).astype(np.float32))
    assert np.array_equal(kp.cpu().numpy(), out.data)


@pytest.mark.parametrize("interleaved,rotary", [(False, 0), (False, 64), (False, 40), (True, 0),
                                                (True, 20)])
@pytest.mark.parametrize("d,group", SHAPES)
def test_rope_append(d, group, interleaved, rotary):
    rotary = min(rotary or d, d)
    rng = np.random.default_rng(rotary + d)
    new, prefix, page, hq, hk = [1, 6, 0, 19], [9, 0, 5, 33], 4, 6, 3
    k, v, app, ptr, idx, last, pool = _append_case(7, new, prefix, page, "NHD", hk, d, group)
    n = int(app[-1])
    x = W.normal_bf16_bits(rng, (n + 2, hq + 2 * hk, d))
    xd = bf16(x)
    f = cache.rope_frequencies(rotary)
    rope = pka.make_rope(rotary, interleaved=interleaved, magnitude=1.2)
    params = pka.make_params(hq, hk, d, page, kv_dtype=_name(group))
    kp, vp = _dev(pool), _dev(pool)
    q_out = torch.zeros(n + 2, hq, d, dtype=torch.bfloat16, device="cuda")
    pka.pka_rope_append_paged_kv_cache(params, rope, xd[:, :hq], q_out, xd[:, hq:hq + hk],
                                       xd[:, hq + hk:], i32(app), i32(ptr), i32(idx), i32(last),
                                       kp, vp, kp.stride(0))
    torch.cuda.synchronize()
    assert pka.pka_get_device_error() == 0 and not q_out[n:].any()
    slots = cache.append_slots(app, ptr, idx, last, page)
    pos = np.array([s[1] for s in slots])
    xf = ref.bf16_bits_to_f64(x[:n])
    turned = cache.rope(xf[:, hq:hq + hk], pos, f, interleaved=interleaved, magnitude=1.2)
    # V is not rotated: exact
    assert np.array_equal(vp.cpu().numpy(),
                          _appended(pool, xf[:, hq + hk:], app, ptr, idx, last))
    got = pool.copy()
    got.data[:] = kp.cpu().numpy()
    want = pool.copy()
    want.data[:] = _appended(pool, turned, app, ptr, idx, last)
    differ = 0
    for row, _, p, s in slots:
        a, b = got.read(p, s), want.read(p, s)
        step = np.repeat(kv4.quantize(turned[row].astype(np.float32), group)[1], group, -1)
        assert np.all(np.abs(a - b) <= step * (1 + 15 * 2.0 ** -7) + 2.0 ** -7 * 1.2 * 8)
        differ += int((a != b).sum())
    # a code or word that differs needs a value within rounding of a border: rare
    assert differ <= 0.01 * n * hk * d
    # untouched bytes: everything but the appended slots
    for row, _, p, s in slots:
        got.write(p, s, np.zeros((hk, d), np.float32))
        want.write(p, s, np.zeros((hk, d), np.float32))
    assert np.array_equal(got.data, want.data)
    qw = cache.rope(xf[:, :hq], pos, f, interleaved=interleaved, magnitude=1.2)
    assert np.all(np.abs(f64(q_out[:n]) - qw) <= 2.0 ** -8 * np.abs(qw) + 2.0 ** -18 * 16)


# ---------------------------------------------------------------------------
# Read-back
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("d,group", SHAPES)
@pytest.mark.parametrize("page,hk,lens", [(1, 1, [1]), (4, 3, [9, 1, 30, 4]), (16, 8, [40, 3])])
def test_read(layout, d, group, page, hk, lens):
    """Whole histories and stretches of them, into padded buffers, K and V and each alone."""
    b = Batch(d + page, lens, page=page, layout=layout, hq=hk, hk=hk, d=d, group=group)
    rng = np.random.default_rng(2)
    begin = np.array([rng.integers(0, n) for n in lens], np.int32)
    count = np.array([rng.integers(0, n - s + 1) for n, s in zip(lens, begin)])
    kp, vp = _dev(b.k), _dev(b.v)
    for at, num in ((None, np.asarray(lens)), (begin, count)):
        ind = np.concatenate([[0], np.cumsum(num)]).astype(np.int32)
        n = int(ind[-1])
        want = []
        for p in (b.k, b.v):
            rows = [kv4.request_rows(p, b.kv_indptr, b.kv_indices, r, int(m))
                    for r, m in enumerate(lens)]
            s = begin if at is not None else np.zeros(len(lens), int)
            rows = [x[s[r]:s[r] + num[r]] for r, x in enumerate(rows)]
            want.append(kv4.bf16_round(np.concatenate(rows).astype(np.float32)))
        for which in ((True, True), (True, False), (False, True)):
            outs = [torch.full((n + 3, hk, d), 7.0, dtype=torch.bfloat16, device="cuda")
                    if w else None for w in which]
            pka.pka_read_paged_kv_cache(b.make_params(), None if at is None else i32(at), i32(ind),
                                        *b.table(), kp, vp, kp.stride(0), *outs)
            torch.cuda.synchronize()
            assert pka.pka_get_device_error() == 0
            for o, w in zip(outs, want):
                if o is not None:
                    assert np.array_equal(f64(o[:n]), w.astype(np.float64))
                    assert (o[n:] == 7.0).all()


@pytest.mark.parametrize("kv,scales", [("bf16", (1, 1)), ("e4m3", (0.37, 2.0))])
@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("d", [64, 128])
def test_read_other_types(kv, scales, layout, d):
    b = W.make_paged_batch(d, [1, 1, 1], [9, 1, 30], page_size=4, layout=layout, hq=3, hk=3, d=d,
                           kv_dtype=kv, k_scale=scales[0], v_scale=scales[1])
    pools = [torch.from_numpy(x).cuda() if kv == "e4m3" else bf16(x) for x in (b.k_pool, b.v_pool)]
    params = pka.make_params(3, 3, d, 4, layout, kv_dtype=kv, k_scale=scales[0],
                             v_scale=scales[1])
    ind = b.kv_lens.cumsum()
    ind = np.concatenate([[0], ind]).astype(np.int32)
    outs = [torch.zeros(int(ind[-1]), 3, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pka.pka_read_paged_kv_cache(params, None, i32(ind), i32(b.kv_indptr), i32(b.kv_indices),
                                i32(b.last_page_len), *pools, pools[0].stride(0), *outs)
    torch.cuda.synchronize()
    for o, x, s in zip(outs, (b.k_pool, b.v_pool), scales):
        rows = np.concatenate([ref.gather_request_kv(
            x, layout=layout, page_size=4, kv_indptr=b.kv_indptr, kv_indices=b.kv_indices, req=r,
            kv_len=int(n)) for r, n in enumerate(b.kv_lens)])
        if kv == "bf16":
            assert np.array_equal(bits_of(o), rows)
        else:
            v = (ref.e4m3_to_f64(rows).astype(np.float32) * np.float32(s)).astype(np.float32)
            assert np.array_equal(f64(o), kv4.bf16_round(v).astype(np.float64))


@pytest.mark.parametrize("kv,layout,hk,bytes_a_slot", [
    ("bf16", "NHD", 32, 8192), ("bf16", "HND", 1, 256), ("e4m3", "NHD", 32, 4096),
    ("e4m3", "HND", 1, 128)])
def test_read_of_pages_over_2_gb(kv, layout, hk, bytes_a_slot):
    """One page a request, past 2 GB: a row's place in it does not fit 32 bits."""
    d, page = 128, (1 << 31) // bytes_a_slot + 70
    shape = (1, page, hk, d) if layout == "NHD" else (1, hk, page, d)
    pool = torch.zeros(shape, dtype=torch.bfloat16 if kv == "bf16" else torch.uint8, device="cuda")
    by_slot = pool if layout == "NHD" else pool.transpose(1, 2)
    begin = np.array([0, page // 2 - 1, page - 70 - 2, page - 3], np.int32)
    g = torch.Generator(device="cuda").manual_seed(hk)
    want = []
    for s in begin:
        if kv == "bf16":
            rows = torch.randn(3, hk, d, generator=g, device="cuda").to(torch.bfloat16)
            by_slot[0, s:s + 3] = rows
        else:
            codes = torch.randint(0, 127, (3, hk, d), generator=g, device="cuda",
                                  dtype=torch.uint8)
            by_slot[0, s:s + 3] = codes
            rows = codes.view(torch.float8_e4m3fn).float().to(torch.bfloat16)
        want.append(rows)
    params = pka.make_params(hk, hk, d, page, layout, kv_dtype=kv)
    n = len(begin)
    outs = [torch.zeros(3 * n, hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pka.pka_read_paged_kv_cache(params, i32(begin), i32(3 * np.arange(n + 1)), i32(np.arange(n + 1)),
                                i32(np.zeros(n)), i32(np.full(n, page)), pool, pool,
                                pool.stride(0), *outs)
    torch.cuda.synchronize()
    assert pka.pka_get_device_error() == 0
    for o in outs:
        assert torch.equal(o, torch.cat(want))


def test_read_steps_around_bad_rows():
    """Positions outside a request's keys and page ids outside the pool are left
    and noted; the other rows come back."""
    b = Batch(4, [9, 6], hq=2, hk=2, d=64, group=32)
    idx = b.kv_indices.copy()
    idx[0], idx[4] = -1, b.k.data.shape[0]  # request 0's first page, request 1's second
    ind, begin = np.array([0, 12, 18], np.int32), np.array([-2, 0], np.int32)
    kp, vp = _dev(b.k), _dev(b.v)
    ko, vo = (torch.full((18, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pka.pka_read_paged_kv_cache(b.make_params(), i32(begin), i32(ind), i32(b.kv_indptr), i32(idx),
                                i32(b.last), kp, vp, kp.stride(0), ko, vo)
    torch.cuda.synchronize()
    assert pka.pka_get_device_error() == 2
    left = list(range(0, 6)) + [11] + [16, 17]
    keep = [i for i in range(18) if i not in left]
    rows = [kv4.request_rows(b.k, b.kv_indptr, b.kv_indices, r, n) for r, n in ((0, 9), (1, 6))]
    want = np.concatenate([rows[0][4:9], rows[1][:4]])
    assert (ko[left] == 7.0).all() and (vo[left] == 7.0).all()
    assert np.array_equal(f64(ko[keep]), kv4.bf16_round(want.astype(np.float32)).astype(float))


def test_nothing_to_do():
    params = pka.make_params(2, 2, 64, 4, kv_dtype="int4_g32")
    pool = torch.zeros(3, pka.pka_kv_page_bytes(params), dtype=torch.uint8, device="cuda")
    none = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    table = [i32(x) for x in ([0, 0], [0, 1], [2], [3])]
    pka.pka_append_paged_kv_cache(params, none, none, *table, pool, pool, pool.stride(0))
    pka.pka_read_paged_kv_cache(params, None, *table, pool, pool, pool.stride(0), none, none)
    one = torch.ones(1, 2, 64, dtype=torch.bfloat16, device="cuda")
    pka.pka_read_paged_kv_cache(params, None, *table, pool, pool, pool.stride(0), one, None)
    torch.cuda.synchronize()
    assert not pool.any() and (one == 1).all() and pka.pka_get_device_error() == 0


# ---------------------------------------------------------------------------
# Attention: decode rows
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("page", [1, 3, 16, 64])
@pytest.mark.parametrize("d,group", SHAPES)
@pytest.mark.parametrize("hq,hk", [(8, 2), (8, 1), (5, 5), (28, 7)])
def test_decode_shapes(layout, page, d, group, hq, hk):
    rng = np.random.default_rng(page * 17 + hq + d)
    kv = rng.integers(1, 400, size=5)
    kv[0] = 1
    b = Batch(int(rng.integers(1 << 30)), kv, page=page, layout=layout, hq=hq, hk=hk, d=d,
              group=group)
    want = b.want()
    for split in (("auto", 1), ("fixed", 2)):
        o, lse, _ = b.run(split_mode=split[0], fixed_split_pages=split[1])
        _assert_decode(o, lse, want)


@pytest.mark.parametrize("n", list(range(1, 18)) + [31, 32, 33, 47, 48, 49, 63, 64, 65, 511, 512,
                                                    513, 1030])
def test_decode_lengths(n):
    b = Batch(n, [n, 1, n + 1], page=16, hq=32, hk=8)
    for split in ("off", "auto"):
        o, lse, _ = b.run(split_mode=split)
        _assert_decode(o, lse, b.want())


@pytest.mark.parametrize("hq,hk", [(64, 8), (32, 32), (12, 12), (16, 16), (24, 3), (6, 6)])
def test_decode_head_counts(hq, hk):
    """Heads in one block and in several, one to sixteen warps a head, groups of one to eight."""
    b = Batch(hq + hk, [77, 300, 5], page=8, hq=hq, hk=hk, d=64, group=64)
    for split in ("off", "auto"):
        o, lse, _ = b.run(split_mode=split)
        _assert_decode(o, lse, b.want())


@pytest.mark.parametrize("spread,q_scale", [(1e-3, 1.0), (300.0, 1.0), (1.0, 2.0 ** -40),
                                            (1.0, 30.0), (1e-12, 1e12)])
def test_decode_magnitudes(spread, q_scale):
    """Small and large K, V and Q, peaked and flat rows: Q's and P's scaling to f16."""
    b = Batch(9, [700, 40, 3], page=16, hq=8, hk=2, group=32, spread=spread)
    b.q = (kv4.bf16_round((ref.bf16_bits_to_f64(b.q) * q_scale).astype(np.float32))
           .view(np.uint32) >> 16).astype(np.uint16)
    o, lse, _ = b.run()
    _assert_decode(o, lse, b.want())


def test_decode_steps_of_all_sizes():
    """V's steps from none (rows of one value) over 2^-100 to 2^12 among the keys of
    one request, the largest late and early."""
    for order in (1, -1):
        b = Batch(10, [260], page=4, hq=4, hk=2, d=64, group=32)
        rng = np.random.default_rng(3)
        size = 2.0 ** np.linspace(-100, 12, 260)[::order]
        for j in range(260):
            row = rng.standard_normal((2, 64)) * size[j]
            if j % 7 == 0:
                row = np.full((2, 64), size[j])
            b.v.write(int(b.kv_indices[j // 4]), j % 4, row.astype(np.float32))
        o, lse, _ = b.run()
        _assert_decode(o, lse, b.want())


@pytest.mark.parametrize("apart", [2.0 ** -12, 2.0 ** -24, 2.0 ** -32, 2.0 ** -60, 2.0 ** -90])
@pytest.mark.parametrize("d,group,hq", [(64, 32, 4), (64, 32, 8), (128, 32, 4), (128, 32, 8),
                                        (128, 64, 4), (128, 64, 8)])
def test_decode_groups_of_unlike_magnitudes(d, group, hq, apart):
    """V's groups of one head far apart in size, one request with the large one first and one
    with it last, and a third where they change places from key to key: each output within
    the bits of what it sums."""
    kv = [70, 300, 130]
    b = Batch(41, kv, page=4, hq=hq, hk=1, d=d, group=group)
    rng = np.random.default_rng(13)
    n = d // group
    sizes = apart ** (np.arange(n) / (n - 1))
    rows = [rng.standard_normal((m, 1, d)) * np.repeat(s, group)
            for m, s in zip(kv, (sizes, sizes[::-1], sizes))]
    rows[2][::2] = rows[2][::2, :, ::-1]
    kv4.fill(b.v, b.kv_indptr, b.kv_indices, b.kv_lens, rows)
    for split in ("off", "auto"):
        o, lse, _ = b.run(split_mode=split)
        _assert_decode(o, lse, b.want())


@pytest.mark.parametrize("order", [1, -1])
def test_decode_weights_against_sizes(order):
    """Keys whose V is the larger the less they weigh, over 2^60: what each adds to an output
    is of one size, however large or small its step."""
    n, d = 240, 64
    b = Batch(42, [n], page=4, hq=4, hk=1, d=d, group=32)
    rng = np.random.default_rng(14)
    sign = np.where(np.arange(d) % 2 == 0, 1.0, -1.0)
    b.q[:] = (np.where(sign > 0, 0x3F80, 0xBF80)).astype(np.uint16)
    weight = np.linspace(-60, 0, n)[::order]  # log2
    k = np.zeros((n, 1, d)) + weight[:, None, None] * sign / (d ** 0.5 * np.log2(np.e))
    v = rng.standard_normal((n, 1, d)) * 2.0 ** -weight[:, None, None]
    for pool, rows in ((b.k, k), (b.v, v)):
        kv4.fill(pool, b.kv_indptr, b.kv_indices, b.kv_lens, [rows])
    for split in ("off", "auto"):
        o, lse, _ = b.run(split_mode=split)
        _assert_decode(o, lse, b.want())


@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** -60, 2.0 ** 40, 2.0 ** 100, 2.0 ** 112])
def test_decode_values_of_any_size(size):
    """V of any size, among it rows of one value, which have no steps; the other request's
    V is of ordinary size."""
    b = Batch(43, [150, 40], page=4, hq=8, hk=2, d=128, group=64)
    rng = np.random.default_rng(15)
    rows = [size * rng.standard_normal((150, 2, 128)), rng.standard_normal((40, 2, 128))]
    rows[0][::5] = size * rng.standard_normal((30, 2, 1))
    kv4.fill(b.v, b.kv_indptr, b.kv_indices, b.kv_lens, rows)
    for split in ("off", "auto"):
        o, lse, _ = b.run(split_mode=split)
        _assert_decode(o, lse, b.want())
    rows[0][:] = size * rng.standard_normal((150, 2, 1))
    kv4.fill(b.v, b.kv_indptr, b.kv_indices, b.kv_lens, rows)
    o, lse, _ = b.run()
    _assert_decode(o, lse, b.want())


@pytest.mark.parametrize("n", [1, 9, 16, 40, 400, 3000])
@pytest.mark.parametrize("d,group,hq", [(64, 32, 4), (64, 64, 8), (128, 32, 8), (128, 64, 4),
                                        (128, 128, 4), (128, 128, 8)])
def test_decode_of_values_from_zero_up(d, group, hq, n):
    """V without negative values, some elements 0 in every key: their outputs are 0 but for
    the sums' own rounding.  An output adds what its second keys' codes lack of 15, so it
    sums magnitudes of at most 15 steps a key, 1.01 here, where an MMA of 16 keys rounds
    2^-23 of its sum (accumulation may truncate), and the few terms beside it as much."""
    b = Batch(44 + n, [n, 33], page=16, hq=hq, hk=1, d=d, group=group)
    rng = np.random.default_rng(16)
    none = np.arange(d) % group % 8 == 3
    rows = [np.where(none, 0.0, rng.random((m, 1, d))) for m in (n, 33)]
    kv4.fill(b.v, b.kv_indptr, b.kv_indices, b.kv_lens, rows)
    want = b.want()
    assert not want[0][..., none].any()
    for split in ("off", "auto"):
        o, lse, _ = b.run(split_mode=split)
        _assert_decode(np.where(none, 0.0, o), lse, want)
        assert np.abs(o[..., none]).max() <= 1.01 * 2.0 ** -22 * (n / 16 + 4)


@pytest.mark.parametrize("hq,hk", [(4, 1), (8, 1)])
def test_long_flat_rows_keep_their_precision(hq, hk):
    """160,000 keys of near equal weight in one piece: the output, the mean of as many
    values, is 400 times smaller than they.  Its own rounding to bf16 is 2^-8 / sqrt(3)
    of it (rms, at most), P's to f16 2^-11 / sqrt(3) of step * code (rms 2.9 values)
    a key, independently, 0.0009 of it; 313 tiles a warp round sums of at most a
    hundredth of the values' own by 2^-23, 0.0002 of it."""
    n = 160000
    rng = np.random.default_rng(60)
    params = pka.make_params(hq, hk, 128, 64, kv_dtype="int4_g128")
    size, pages = pka.pka_kv_page_bytes(params), n // 64
    pools = [torch.zeros(pages, size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    g = torch.Generator(device="cuda").manual_seed(6)
    rows = [torch.randn(n, hk, 128, generator=g, device="cuda").to(torch.bfloat16)
            for _ in range(2)]
    ptr, idx = np.array([0, pages], np.int32), rng.permutation(pages).astype(np.int32)
    last = np.array([64], np.int32)
    pka.pka_append_paged_kv_cache(params, *rows, i32([0, n]), i32(ptr), i32(idx), i32(last),
                                  *pools, size)
    q = W.normal_bf16_bits(rng, (1, hq, 128))
    q = (kv4.bf16_round((ref.bf16_bits_to_f64(q) / 64).astype(np.float32)).view(np.uint32)
         >> 16).astype(np.uint16)
    attn = pka.BatchAttention()
    attn.plan(None, ptr, last, num_qo_heads=hq, num_kv_heads=hk, head_dim=128, page_size=64,
              split_mode="off", kv_dtype="int4_g128")
    o, _ = attn.run(bf16(q), *pools, i32(idx))
    torch.cuda.synchronize()
    kp, vp = (kv4.Pool(p.cpu().numpy(), 64, hk, 128, 128, "NHD") for p in pools)
    want = kv4.attention(q, kp, vp, qo_indptr=[0, 1], kv_indptr=ptr, kv_indices=idx, kv_lens=[n],
                         hq=hq, hk=hk)[0]
    rel = np.sqrt(((f64(o) - want) ** 2).mean() / (want ** 2).mean())
    assert rel <= 2.0 ** -8 / np.sqrt(3) + 0.0009 + 0.0002


def test_decode_zero_query_and_queries_of_zeros_and_one_value():
    b = Batch(11, [50, 20], page=16, hq=8, hk=2, group=64)
    b.q[0] = 0
    b.q[1, :, 1:] = 0
    o, lse, _ = b.run()
    _assert_decode(o, lse, b.want())
    assert np.allclose(lse[0], np.log2(50), atol=1e-5)


def test_decode_full_size():
    """The benchmark's batch decode: 64 requests of 512..4096 keys, split over every SM."""
    rng = np.random.default_rng(1001)
    kv = rng.integers(512, 4096, size=64, endpoint=True)
    g = torch.Generator(device="cuda").manual_seed(5)
    params = pka.make_params(32, 8, 128, 16, kv_dtype="int4_g128")
    ptr, idx, last, pages = W.build_page_table(rng, kv, 16)
    size = pka.pka_kv_page_bytes(params)
    pools = [torch.zeros(pages, size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    n = int(kv.sum())
    rows = [torch.randn(n, 8, 128, generator=g, device="cuda").to(torch.bfloat16)
            for _ in range(2)]
    app = np.concatenate([[0], np.cumsum(kv)]).astype(np.int32)
    table = (i32(ptr), i32(idx), i32(last))
    pka.pka_append_paged_kv_cache(params, *rows, i32(app), *table, *pools, size)
    b = Batch(12, [1], page=16, hq=32, hk=8)
    b.kv_lens, b.kv_indptr, b.kv_indices, b.last = kv, ptr, idx, last
    b.qo_indptr = np.arange(65, dtype=np.int32)
    b.q = W.normal_bf16_bits(rng, (64, 32, 128))
    b.k, b.v = (kv4.Pool(p.cpu().numpy(), 16, 8, 128, 128, "NHD") for p in pools)
    o, lse, info = b.run()
    assert info.num_decode_joins > 0
    _assert_decode(o, lse, b.want())


def test_decode_custom_masks():
    """Masked keys, a row that sees none, and NaN and infinities in what is masked."""
    b = Batch(13, [70, 40, 33, 1], page=4, hq=8, hk=2, group=64)
    rng = np.random.default_rng(4)
    mask = [rng.random(70) < 0.5, np.zeros(40, bool), np.arange(33) == 32, np.ones(1, bool)]
    for j in np.nonzero(~mask[0])[0][:20]:
        row = np.full((2, 128), np.nan if j % 2 else np.inf, np.float32)
        for p in (b.k, b.v):
            p.write(int(b.kv_indices[j // 4]), j % 4, row)
    flat = np.concatenate(mask)
    packed = torch.from_numpy(np.packbits(flat, bitorder="little")).cuda()
    clean = Batch(13, [70, 40, 33, 1], page=4, hq=8, hk=2, group=64)
    want = clean.want(mask="custom", mask_bool=flat)
    for split in (("auto", 1), ("fixed", 3)):
        o, lse, _ = b.run(mask=packed, mask_mode="custom", split_mode=split[0],
                          fixed_split_pages=split[1])
        _assert_decode(o, lse, want)
        assert not o[1].any() and np.all(lse[1] == -np.inf)


@pytest.mark.parametrize("which", ["k", "v"])
def test_nan_group_shows(which):
    """A seen key whose group is NaN makes the outputs NaN that it reaches: every
    element through K, its own group's through V; other requests stay as they were."""
    b = Batch(14, [50, 20], page=4, hq=4, hk=2, d=128, group=32)
    clean = b.want()
    row = np.ones((2, 128), np.float32)
    row[0, 40] = np.nan  # head 0, group 1
    getattr(b, which).write(int(b.kv_indices[2]), 1, row)
    o, lse, _ = b.run()
    hit = slice(0, 128) if which == "k" else slice(32, 64)
    assert np.isnan(o[0, :2, hit]).all()
    assert np.isnan(lse[0, :2]).all() == (which == "k")
    if which == "v":
        assert np.isfinite(o[0, :2, :32]).all() and np.isfinite(o[0, :2, 64:]).all()
    assert np.isfinite(o[0, 2:]).all()
    _assert_decode(o, lse, clean, rows=[1])


@pytest.mark.parametrize("splits", ["off", "auto"])
def test_run_again_and_on_another_stream(splits):
    """One plan, several runs, on two streams one after the other: the same bits."""
    b = Batch(15, [3000, 10, 900], page=16, hq=32, hk=8)
    attn = pka.BatchAttention()
    attn.plan(b.qo_indptr, b.kv_indptr, b.last, **b.params(split_mode=splits))
    q, k, v, idx = bf16(b.q), _dev(b.k), _dev(b.v), i32(b.kv_indices)
    first = attn.run(q, k, v, idx)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = attn.run(q, k, v, idx, stream=side, out=torch.empty_like(q))
    torch.cuda.current_stream().wait_stream(side)
    third = attn.run(q, k, v, idx)
    torch.cuda.synchronize()
    _assert_decode(f64(first[0]), f64(first[1]), b.want())
    for o, lse in (again, third):  # pieces may merge in another order of arrival, not of sums
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])


def test_strided_pools_and_page_padding():
    """K and V in one allocation, 5 pages apart, and pages whose words end off a
    multiple of 16 bytes."""
    b = Batch(16, [20, 7], page=1, hq=1, hk=1, d=128, group=128)
    n, size = b.k.data.shape
    assert size == 80  # 68 bytes of codes and word, padded
    both = torch.full((n, 5, size), 0xEE, dtype=torch.uint8, device="cuda")
    both[:, 1], both[:, 3] = _dev(b.k), _dev(b.v)
    attn = pka.BatchAttention()
    attn.plan(b.qo_indptr, b.kv_indptr, b.last, **b.params())
    o, lse = attn.run(bf16(b.q), both[:, 1], both[:, 3], i32(b.kv_indices))
    torch.cuda.synchronize()
    _assert_decode(f64(o), f64(lse), b.want())


def test_far_pages():
    """A page whose bytes lie past 2^32 in the pool."""
    b = Batch(17, [40, 90], page=16, hq=8, hk=2, d=128, group=64)
    size = b.k.data.shape[1]
    far = (1 << 32) // size + 5
    n = b.k.data.shape[0]
    pools = []
    for p in (b.k, b.v):
        t = torch.zeros(far + n, size, dtype=torch.uint8, device="cuda")
        t[far:] = _dev(p)
        pools.append(t)
    attn = pka.BatchAttention()
    attn.plan(b.qo_indptr, b.kv_indptr, b.last, **b.params())
    o, lse = attn.run(bf16(b.q), *pools, i32(b.kv_indices + far))
    ind = np.concatenate([[0], np.cumsum(b.kv_lens)]).astype(np.int32)
    ko = torch.zeros(130, 2, 128, dtype=torch.bfloat16, device="cuda")
    table = (i32(b.kv_indptr), i32(b.kv_indices + far), i32(b.last))
    pka.pka_read_paged_kv_cache(b.make_params(), None, i32(ind), *table, *pools, size, ko)
    before = pools[0][far:].clone()
    pka.pka_append_paged_kv_cache(b.make_params(), ko, ko, i32(ind), *table, *pools, size)
    torch.cuda.synchronize()
    _assert_decode(f64(o), f64(lse), b.want())
    want = np.concatenate([kv4.request_rows(b.k, b.kv_indptr, b.kv_indices, r, int(m))
                           for r, m in enumerate(b.kv_lens)])
    assert np.array_equal(f64(ko), kv4.bf16_round(want.astype(np.float32)).astype(float))
    assert not torch.equal(pools[1][far:], _dev(b.v)) and not pools[0][:far].any()
    assert before.shape == pools[0][far:].shape and pka.pka_get_device_error() == 0


# ---------------------------------------------------------------------------
# Rows through the f16 scratch, cascades, captured runs
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("page", [1, 3, 16])
@pytest.mark.parametrize("d,group", SHAPES)
def test_mixed_rows(layout, page, d, group):
    """Decode rows and rows with qo_len >= 2 in one batch, all in one run."""
    qo, kv = [1, 5, 130, 0, 1, 2], [77, 60, 300, 4, 1, 2]
    b = Batch(page + d, kv, qo_lens=qo, page=page, layout=layout, hq=8, hk=2, d=d, group=group)
    o, lse, info = b.run()
    assert info.kv_scratch_rows == 60 + 300 + 2
    want = b.want()
    _assert_staged(o, lse, want, rows=list(range(1, 136)) + [137, 138])
    _assert_decode(o, lse, want, rows=[0, 136])


@pytest.mark.parametrize("hq,hk", [(5, 5), (8, 1), (28, 7), (32, 4)])
def test_rows_and_head_counts(hq, hk):
    b = Batch(hq, [200, 9, 33], qo_lens=[140, 3, 2], page=16, hq=hq, hk=hk, d=64, group=32)
    for kw in (dict(), dict(mask_mode="none"), dict(split_mode="fixed", fixed_split_pages=2)):
        o, lse, _ = b.run(**kw)
        _assert_staged(o, lse, b.want(mask=kw.get("mask_mode", "causal")))


@pytest.mark.parametrize("k_size,v_size,q_size", [(1e-4, 1e-6, 1.0), (300.0, 5000.0, 0.01),
                                                  (2.0 ** 40, 2.0 ** 60, 2.0 ** -40),
                                                  (2.0 ** -60, 2.0 ** -70, 2.0 ** 30), (0, 0, 0)])
def test_staged_magnitudes(k_size, v_size, q_size):
    """K, V and Q of any size, one request's a 2^-12th of the other's, and all zeros."""
    b = Batch(20, [90, 70], qo_lens=[40, 7], page=4, hq=8, hk=2, d=64, group=32)
    rng = np.random.default_rng(8)
    for pool, size in ((b.k, k_size), (b.v, v_size)):
        rows = [size * (2.0 ** -12 if r else 1) * rng.standard_normal((n, 2, 64))
                for r, n in enumerate((90, 70))]
        kv4.fill(pool, b.kv_indptr, b.kv_indices, b.kv_lens, rows)
    x = (ref.bf16_bits_to_f64(b.q) * q_size).astype(np.float32)
    b.q = (kv4.bf16_round(x).view(np.uint32) >> 16).astype(np.uint16)
    o, lse, _ = b.run()
    want = b.want()
    _assert_staged(o, lse, want)


@pytest.mark.parametrize("apart", [2.0 ** 45, 2.0 ** 60])
@pytest.mark.parametrize("rows", [(40, 7), (2, 1)])
def test_staged_requests_of_unlike_magnitudes(apart, rows):
    """Requests of one launch whose K and V are 2^45 or 2^60 apart, the large one first, in
    the middle and last: each has the bits that it has alone."""
    kv = [90, 70, 129]
    for large in range(3):
        size = [apart if r == large else 1.0 for r in range(3)]
        b = Batch(26, kv, qo_lens=[rows[0], rows[1], 3], page=4, hq=8, hk=2, d=64, group=32)
        rng = np.random.default_rng(8)
        x = ref.bf16_bits_to_f64(b.q)
        for r in range(3):
            x[b.qo_indptr[r]:b.qo_indptr[r + 1]] /= size[r]
        b.q = (kv4.bf16_round(x.astype(np.float32)).view(np.uint32) >> 16).astype(np.uint16)
        for pool in (b.k, b.v):
            kv4.fill(pool, b.kv_indptr, b.kv_indices, b.kv_lens,
                     [s * rng.standard_normal((n, 2, 64)) for s, n in zip(size, kv)])
        kw = dict(decode_on_tensor_cores=True)
        o, lse, info = b.run(**kw)
        assert info.kv_scratch_rows == sum(kv)
        _assert_staged(o, lse, b.want())
        for r in range(3):
            q0, q1 = b.qo_indptr[r], b.qo_indptr[r + 1]
            p0, p1 = b.kv_indptr[r], b.kv_indptr[r + 1]
            attn = pka.BatchAttention()
            attn.plan(np.array([0, q1 - q0], np.int32), np.array([0, p1 - p0], np.int32),
                      b.last[r:r + 1], **b.params(mask_mode="causal", **kw))
            alone, alone_lse = attn.run(bf16(b.q[q0:q1]), _dev(b.k), _dev(b.v),
                                        i32(b.kv_indices[p0:p1]))
            torch.cuda.synchronize()
            assert np.array_equal(f64(alone), o[q0:q1])
            assert np.array_equal(f64(alone_lse), lse[q0:q1])


def test_custom_masks_of_several_rows():
    """Masks of several rows; what they hide may be NaN, in K and in V."""
    qo, kv = [3, 1, 9], [40, 20, 33]
    b, clean = (Batch(21, kv, qo_lens=qo, page=4, hq=8, hk=2, d=64, group=64) for _ in range(2))
    rng = np.random.default_rng(6)
    masks = [rng.random((a, c)) < 0.4 for a, c in zip(qo, kv)]
    masks[2][4] = False  # a row that sees nothing
    masks[0][:, 7], masks[2][:, 30] = False, False
    for pool, r, j in ((b.k, 0, 7), (b.v, 0, 7), (b.v, 2, 30)):
        pool.write(int(b.kv_indices[b.kv_indptr[r] + j // 4]), j % 4,
                   np.full((2, 64), np.nan, np.float32))
    flat = np.concatenate([m.reshape(-1) for m in masks])
    packed = torch.from_numpy(np.packbits(flat, bitorder="little")).cuda()
    want = clean.want(mask="custom", mask_bool=flat)
    for split in (("auto", 1), ("fixed", 2)):
        o, lse, _ = b.run(mask=packed, mask_mode="custom", split_mode=split[0],
                          fixed_split_pages=split[1])
        _assert_staged(o, lse, want, rows=[0, 1, 2] + list(range(4, 13)))
        _assert_decode(o, lse, want, rows=[3])
        assert not o[8].any() and np.all(lse[8] == -np.inf)


@pytest.mark.parametrize("which", ["k", "v"])
def test_staged_nan_group_shows(which):
    """A NaN group makes the rows that see it NaN, and neither the rows before it nor
    the request whose staged keys lie beside it."""
    b = Batch(24, [60, 40], qo_lens=[20, 30], page=4, hq=4, hk=2, d=128, group=32)
    clean = b.want()
    row = np.ones((2, 128), np.float32)
    row[0, 40] = np.nan
    j = 50  # seen by request 0's rows from 10 on, in kv head 0
    getattr(b, which).write(int(b.kv_indices[j // 4]), j % 4, row)
    getattr(clean_other := Batch(24, [60, 40], qo_lens=[20, 30], page=4, hq=4, hk=2, d=128,
                                 group=32), which).write(
        int(b.kv_indices[j // 4]), j % 4, np.where(np.isnan(row), 1, row))
    o, lse, _ = b.run()
    hit = slice(0, 128) if which == "k" else slice(32, 64)
    assert np.isnan(o[10:20, :2, hit]).all() and np.isnan(lse[10:20, :2]).all()
    other = clean_other.want()
    _assert_staged(o, lse, clean, rows=list(range(0, 10)) + list(range(20, 50)))
    for x in (o, lse):
        assert np.isfinite(x[10:20, 2:]).all()
    _assert_staged(o[10:20, 2:], lse[10:20, 2:], tuple(x[10:20, 2:] for x in other))


@pytest.mark.parametrize("apart", [2.0 ** 13, 2.0 ** 18, 2.0 ** 24, 2.0 ** 40, 2.0 ** 100])
@pytest.mark.parametrize("which", ["k", "v", "both"])
def test_staged_keys_behind_a_mask_of_any_size(apart, which):
    """Finite keys that a mask hides, the request's last ones (behind most rows' causal
    ends, too) and one in the middle, far larger than those that are seen."""
    qo, kv = [6, 1, 9], [140, 60, 33]
    b = Batch(29, kv, qo_lens=qo, page=4, hq=8, hk=2, d=64, group=32)
    rng = np.random.default_rng(9)
    masks = [rng.random((a, c)) < 0.7 for a, c in zip(qo, kv)]
    masks[2][4] = False  # a row that sees nothing
    hide = [(0, 7), (0, 138), (0, 139), (1, 30), (2, 0), (2, 32)]
    for r, j in hide:
        masks[r][:, j] = False
        for pool in {"k": (b.k,), "v": (b.v,), "both": (b.k, b.v)}[which]:
            pool.write(int(b.kv_indices[b.kv_indptr[r] + j // 4]), j % 4,
                       (apart * rng.standard_normal((2, 64))).astype(np.float32))
    flat = np.concatenate([m.reshape(-1) for m in masks])
    packed = torch.from_numpy(np.packbits(flat, bitorder="little")).cuda()
    o, lse, _ = b.run(mask=packed, mask_mode="custom")
    want = b.want(mask="custom", mask_bool=flat)
    check = _assert_staged if apart < 2.0 ** 16 else _assert_wide
    check(o, lse, want, rows=[0, 1, 2, 3, 4, 5] + list(range(7, 16)))
    _assert_decode(o, lse, want, rows=[6])
    assert not o[11].any() and np.all(lse[11] == -np.inf)


def test_staged_keys_behind_the_causal_end_of_any_size():
    """Chunks over a prefix, the last key of each request 2^60 of the others: the rows
    before the last do not see it."""
    qo, kv = [130, 5, 300], [300, 77, 300]
    b = Batch(30, kv, qo_lens=qo, page=16, hq=8, hk=2, d=128, group=64)
    rng = np.random.default_rng(10)
    for r, n in enumerate(kv):
        for pool in (b.k, b.v):
            pool.write(int(b.kv_indices[b.kv_indptr[r] + (n - 1) // 16]), (n - 1) % 16,
                       (2.0 ** 60 * rng.standard_normal((2, 128))).astype(np.float32))
    o, lse, _ = b.run()
    last = set(int(x) - 1 for x in b.qo_indptr[1:])
    _assert_wide(o, lse, b.want(), rows=[i for i in range(435) if i not in last])


@pytest.mark.parametrize("apart", [2.0 ** -13, 2.0 ** -19, 2.0 ** -30, 2.0 ** -60])
def test_staged_groups_of_unlike_magnitudes(apart):
    """V's groups of one head, and the keys of one request, far apart in size and all seen:
    each output within the bits of what it sums."""
    b = Batch(31, [150, 90], qo_lens=[20, 4], page=4, hq=8, hk=2, d=128, group=32)
    rng = np.random.default_rng(11)
    sizes = np.repeat([1.0, apart, apart ** 0.5, apart], 32)
    rows = [rng.standard_normal((n, 2, 128)) * sizes for n in (150, 90)]
    rows[1][::3, :, 32:64] *= 0  # groups of zeros are of no size
    kv4.fill(b.v, b.kv_indptr, b.kv_indices, b.kv_lens, rows)
    o, lse, _ = b.run()
    (_assert_staged if apart > 2.0 ** -16 else _assert_wide)(o, lse, b.want())


def test_staged_keys_of_all_sizes():
    """V's keys from none over 2^-100 to 2^12 within a request, as decode rows take them."""
    for order in (1, -1):
        b = Batch(10, [260], qo_lens=[200], page=4, hq=4, hk=2, d=64, group=32)
        rng = np.random.default_rng(3)
        size = 2.0 ** np.linspace(-100, 12, 260)[::order]
        for j in range(260):
            row = rng.standard_normal((2, 64)) * size[j]
            if j % 7 == 0:
                row = np.full((2, 64), size[j])
            b.v.write(int(b.kv_indices[j // 4]), j % 4, row.astype(np.float32))
        o, lse, _ = b.run()
        _assert_wide(o, lse, b.want())


def _set_word(pool, page, slot, head, group, step, origin):
    """A word of the pool from the bits of its step and origin."""
    n = pool.D // pool.g
    at = pool.P * pool.H * (pool.D // 2) + (pool._row(slot, head) * n + group) * 4
    pool.data[page, at:at + 4] = np.array([step, origin], np.uint16).view(np.uint8)


INF, LARGE = 0x7F80, 0x7F7F  # bits of bf16 infinity and of its largest number


@pytest.mark.parametrize("step,origin", [(0, INF), (0, INF | 0x8000), (INF, 0), (INF, INF | 0x8000),
                                         (LARGE, LARGE), (0x7FC0, 0), (0x3F80, 0x7FC0)])
def test_words_that_are_not_finite(step, origin):
    """Infinite words (or whose 16th value is past float32), in V's and in K's groups: the
    rows that see one are not finite, the rows that do not, by their causal end or in
    another request, keep their values."""
    qo, kv = [20, 30, 1], [60, 40, 25]
    for hidden in (True, False):
        b, clean = (Batch(27, kv, qo_lens=qo, page=4, hq=4, hk=2, d=128, group=64)
                    for _ in range(2))
        j, r = (59, 0) if hidden else (50, 0)  # seen by the last row alone, or from row 10 on
        for pool in (b.v,) if hidden else (b.k, b.v):
            _set_word(pool, int(b.kv_indices[b.kv_indptr[r] + j // 4]), j % 4, 0, 1, step, origin)
        want = clean.want()
        o, lse, _ = b.run()
        first = 19 if hidden else 10
        _assert_staged(o, lse, want, rows=list(range(first)) + list(range(20, 50)))
        _assert_decode(o, lse, want, rows=[50])
        assert np.isfinite(o[first:20, 2:]).all()
        assert not np.isfinite(o[first:20, :2, 64:]).any()


def test_infinite_words_behind_a_mask():
    """A mask's hidden keys may be infinite in V, for staged rows and for decode rows."""
    qo, kv = [5, 1], [40, 30]
    b, clean = (Batch(28, kv, qo_lens=qo, page=4, hq=8, hk=2, d=64, group=32) for _ in range(2))
    masks = [np.ones((a, c), bool) for a, c in zip(qo, kv)]
    for r, j in ((0, 7), (0, 39), (1, 3)):
        masks[r][:, j] = False
        for h in range(2):
            _set_word(b.v, int(b.kv_indices[b.kv_indptr[r] + j // 4]), j % 4, h, 1, 0, INF)
    flat = np.concatenate([m.reshape(-1) for m in masks])
    packed = torch.from_numpy(np.packbits(flat, bitorder="little")).cuda()
    want = clean.want(mask="custom", mask_bool=flat)
    o, lse, _ = b.run(mask=packed, mask_mode="custom")
    _assert_staged(o, lse, want, rows=list(range(5)))
    _assert_decode(o, lse, want, rows=[5])


@pytest.mark.parametrize("below", [14.0, 20.0, 24.6, 25.2, 27.0, 31.0])
def test_staged_long_tails(below):
    """131,072 keys of one weight, 2^-14 to 2^-31 of the first key's, whose V is 0: the output
    is all theirs, and none of it may be lost in P's rounding."""
    n, hq, hk, d = 131073, 4, 1, 64
    params = pka.make_params(hq, hk, d, 64, kv_dtype="int4_g32")
    size, pages = pka.pka_kv_page_bytes(params), -(-n // 64)
    pools = [torch.zeros(pages, size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    g = torch.Generator(device="cuda").manual_seed(7)
    sign = torch.where(torch.arange(d, device="cuda") % 2 == 0, 1.0, -1.0)
    k = torch.zeros(n, hk, d, device="cuda")
    k[0] = sign * (below / (d ** 0.5 * np.log2(np.e)))  # q . k / sqrt(d) in log2 units
    v = torch.rand(n, hk, d, generator=g, device="cuda") + 0.5
    v[0] = 0
    ptr, idx = np.array([0, pages], np.int32), np.arange(pages, dtype=np.int32)
    last = np.array([n - (pages - 1) * 64], np.int32)
    pka.pka_append_paged_kv_cache(params, k.to(torch.bfloat16), v.to(torch.bfloat16), i32([0, n]),
                                  i32(ptr), i32(idx), i32(last), *pools, size)
    q = sign.expand(2, hq, d).contiguous().to(torch.bfloat16)
    attn = pka.BatchAttention()
    attn.plan(np.array([0, 2], np.int32), ptr, last, num_qo_heads=hq, num_kv_heads=hk, head_dim=d,
              page_size=64, mask_mode="none", split_mode="off", kv_dtype="int4_g32")
    o, lse = attn.run(q, *pools, i32(idx))
    torch.cuda.synchronize()
    kp, vp = (kv4.Pool(p.cpu().numpy(), 64, hk, d, 32, "NHD") for p in pools)
    want = kv4.attention(bits_of(q), kp, vp, qo_indptr=[0, 2], kv_indptr=ptr, kv_indices=idx,
                         kv_lens=[n], hq=hq, hk=hk, mask="none")
    # the scores: 64 products of one size, exact in K's bits but for its rounding to f16, which
    # moves all of them as one: 2^-11 of the score
    shift = 2.0 ** -11 * below
    assert np.abs(f64(lse) - want[1]).max() <= shift + 2.0 ** -17
    tail = 2.0 ** -36 * 1.5 * (n - 1)
    tol = (2 * np.log(2) * 2 * shift + 2 * 2.0 ** -11 + 2.0 ** -13 + 2.0 ** -8) * want[0] + tail
    assert np.all(np.abs(f64(o) - want[0]) <= tol)


def test_decode_on_tensor_cores():
    b = Batch(22, [90, 1, 400], page=16, hq=8, hk=2, group=64)
    o, lse, info = b.run(decode_on_tensor_cores=True)
    assert info.num_decode_items == 0 and info.kv_scratch_rows == 491
    _assert_staged(o, lse, b.want())


def test_static_scratch():
    b = Batch(23, [1500, 60], page=16, hq=32, hk=8)
    attn = pka.BatchAttention()
    attn.plan(b.qo_indptr, b.kv_indptr, b.last, **b.params())
    q, k, v = bf16(b.q), _dev(b.k), _dev(b.v)
    o, lse = torch.empty_like(q), torch.empty(2, 32, device="cuda")
    pka.pka_run_static_scratch(attn.handle, attn.params, q, k, v, k.stride(0), i32(b.kv_indices),
                               None, o, lse)
    torch.cuda.synchronize()
    _assert_decode(f64(o), f64(lse), b.want())


@pytest.mark.parametrize("kv_group", [32, 128])
def test_cascade(kv_group):
    """Decode rows under a shared prefix equal the flat batch whose tables list the
    prefix's pages."""
    page, prefix, own = 16, 160, [33, 1, 70, 16]
    kv = [prefix + n for n in own]
    b = Batch(25, kv, page=page, hq=8, hk=2, group=kv_group)
    # every request's first pages are request 0's
    shared = b.kv_indices[:prefix // page].copy()
    for r in range(4):
        b.kv_indices[b.kv_indptr[r]:b.kv_indptr[r] + prefix // page] = shared
    own_pages = [b.kv_indices[b.kv_indptr[r] + prefix // page:b.kv_indptr[r + 1]] for r in range(4)]
    own_ptr = np.concatenate([[0], np.cumsum([len(x) for x in own_pages])]).astype(np.int32)
    levels = [(np.array([0, 4], np.int32), np.array([0, prefix // page], np.int32),
               np.array([page], np.int32)),
              (np.arange(5, dtype=np.int32), own_ptr, b.last)]
    attn = pka.BatchAttention()
    kw = b.params()
    info = attn.plan_cascade(levels, **kw)
    assert info.kv_scratch_rows == prefix  # the root's rows go through the tensor cores
    o, lse = attn.run(bf16(b.q), _dev(b.k), _dev(b.v),
                      i32(np.concatenate([shared] + own_pages)))
    torch.cuda.synchronize()
    _assert_staged(f64(o), f64(lse), b.want())


@pytest.mark.parametrize("rows", ["decode", "mixed"])
def test_graph_replayed_over_plans(rows):
    """One captured run serves later plans of other batches."""
    cap = dict(graph_max_batch=6, graph_max_qo_rows=64, graph_max_kv_tokens=4096)
    attn = pka.BatchAttention()
    size, pages = None, 600
    stream = torch.cuda.Stream()
    graph, hold = None, {}
    for i in range(4):
        rng = np.random.default_rng(30 + i)
        n = [6, 1, 4, 2][i]
        kv = rng.integers(1, 700, n)
        qo = np.ones(n, int)
        if rows == "mixed":
            qo = rng.integers(1, 9, n)
            kv = np.maximum(kv, qo)
        b = Batch(40 + i, kv, qo_lens=qo, page=8, hq=8, hk=2, d=64, group=32)
        size = b.k.data.shape[1]
        if graph is None:
            hold = dict(q=torch.zeros(64, 8, 64, dtype=torch.bfloat16, device="cuda"),
                        o=torch.zeros(64, 8, 64, dtype=torch.bfloat16, device="cuda"),
                        lse=torch.zeros(64, 8, device="cuda"),
                        k=torch.zeros(pages, size, dtype=torch.uint8, device="cuda"),
                        v=torch.zeros(pages, size, dtype=torch.uint8, device="cuda"),
                        idx=torch.zeros(pages, dtype=torch.int32, device="cuda"))
        m = b.k.data.shape[0]
        hold["k"][:m], hold["v"][:m] = _dev(b.k), _dev(b.v)
        hold["idx"][:len(b.kv_indices)] = i32(b.kv_indices)
        hold["q"][:len(b.q)] = bf16(b.q)
        torch.cuda.synchronize()
        pka.pka_plan_wait(attn.handle)
        attn.plan(b.qo_indptr, b.kv_indptr, b.last, stream=stream, **b.params(**cap))

        def call():
            attn.run(hold["q"], hold["k"], hold["v"], hold["idx"], out=hold["o"], lse=hold["lse"],
                     stream=stream)
        if graph is None:
            call()
            stream.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                call()
        with torch.cuda.stream(stream):
            graph.replay()
        stream.synchronize()
        assert pka.pka_get_device_error() == 0
        o, lse = f64(hold["o"][:len(b.q)]), f64(hold["lse"][:len(b.q)])
        one = [int(b.qo_indptr[r]) for r in range(n) if qo[r] == 1]
        more = [i for i in range(len(b.q)) if i not in one]
        _assert_decode(o, lse, b.want(), rows=one)
        _assert_staged(o, lse, b.want(), rows=more)


def test_graph_replayed_over_magnitudes():
    """A captured run takes what the pools hold when it is replayed: groups alike (f16 rows),
    then one request's far apart (its rows in bf16, the others' in f16), then alike again."""
    kv, qo = [150, 40, 77], [9, 3, 1]
    b = Batch(33, kv, qo_lens=qo, page=8, hq=8, hk=2, d=64, group=32)
    attn, stream = pka.BatchAttention(), torch.cuda.Stream()
    cap = dict(graph_max_batch=4, graph_max_qo_rows=20, graph_max_kv_tokens=400)
    q, k, v, idx = bf16(b.q), _dev(b.k), _dev(b.v), i32(b.kv_indices)
    q = torch.cat([q, torch.zeros(7, 8, 64, dtype=torch.bfloat16, device="cuda")])
    o, lse = torch.empty_like(q), torch.empty(20, 8, device="cuda")
    torch.cuda.synchronize()
    attn.plan(b.qo_indptr, b.kv_indptr, b.last, stream=stream, mask_mode="causal",
              **b.params(**cap))
    attn.run(q, k, v, idx, out=o, lse=lse, stream=stream)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        attn.run(q, k, v, idx, out=o, lse=lse, stream=stream)
    rng = np.random.default_rng(12)
    for apart in (1.0, 2.0 ** 40, 1.0):
        sizes = np.repeat([1.0, apart], 32)
        rows = [rng.standard_normal((n, 2, 64)) * (sizes if r == 0 else 1.0)
                for r, n in enumerate(kv)]
        kv4.fill(b.v, b.kv_indptr, b.kv_indices, b.kv_lens, rows)
        v.copy_(_dev(b.v))
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graph.replay()
        stream.synchronize()
        want, got = b.want(), (f64(o[:13]), f64(lse[:13]))
        (_assert_wide if apart > 1 else _assert_staged)(*got, want, rows=list(range(9)))
        _assert_staged(*got, want, rows=[9, 10, 11])
        _assert_decode(*got, want, rows=[12])
    assert pka.pka_get_device_error() == 0


def test_graph_of_decode_rows_alone():
    """Without graph_max_kv_tokens a graph serves decode batches; others are refused."""
    cap = dict(graph_max_batch=5, graph_max_qo_rows=5)
    attn, stream, graph = pka.BatchAttention(), torch.cuda.Stream(), None
    for i, n in enumerate([5, 2, 4]):
        b = Batch(60 + i, np.random.default_rng(i).integers(1, 900, n), page=16, hq=16, hk=2,
                  layout="HND")
        with torch.cuda.stream(stream):
            if graph is None:
                size = b.k.data.shape[1]
                k, v = (torch.zeros(400, size, dtype=torch.uint8, device="cuda") for _ in range(2))
                q, o = (torch.zeros(5, 16, 128, dtype=torch.bfloat16, device="cuda")
                        for _ in range(2))
                lse, idx = torch.zeros(5, 16, device="cuda"), i32(np.zeros(400, np.int32))
            k[:len(b.k.data)], v[:len(b.k.data)] = _dev(b.k), _dev(b.v)
            idx[:len(b.kv_indices)] = i32(b.kv_indices)
            q[:n] = bf16(b.q)
            stream.synchronize()
            pka.pka_plan_wait(attn.handle)
            attn.plan(b.qo_indptr, b.kv_indptr, b.last, stream=stream, **b.params(**cap))
            if graph is None:
                attn.run(q, k, v, idx, out=o, lse=lse, stream=stream)
                stream.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=stream):
                    attn.run(q, k, v, idx, out=o, lse=lse, stream=stream)
            graph.replay()
            stream.synchronize()
        assert pka.pka_get_device_error() == 0
        _assert_decode(f64(o[:n]), f64(lse[:n]), b.want())
    with pytest.raises(pka.PkaError):
        attn.plan(np.array([0, 2], np.int32), b.kv_indptr[:2], b.last[:1], **b.params(**cap))


@pytest.mark.parametrize("hk", [24, 33])
@pytest.mark.parametrize("d,group", SHAPES)
def test_many_heads(d, group, hk):
    """More heads than a warp's lanes take in one go, in pages a stride apart: append,
    read, decode."""
    rng = np.random.default_rng(hk)
    kv = np.array([37, 3, 64])
    ptr, idx, last, pages = W.build_page_table(rng, kv, 16, pool_pages=9)
    ind = np.concatenate([[0], np.cumsum(kv)]).astype(np.int32)
    n = int(ind[-1])
    params = pka.make_params(hk, hk, d, 16, "HND", kv_dtype=_name(group))
    size = pka.pka_kv_page_bytes(params)
    both = torch.full((pages, 3, size), 0x5A, dtype=torch.uint8, device="cuda")
    kp, vp = both[:, 0], both[:, 2]
    k, v = (W.normal_bf16_bits(rng, (n, hk, d)) for _ in range(2))
    table = (i32(ptr), i32(idx), i32(last))
    pka.pka_append_paged_kv_cache(params, bf16(k), bf16(v), i32(ind), *table, kp, vp, kp.stride(0))
    outs = [torch.zeros(n, hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pka.pka_read_paged_kv_cache(params, None, i32(ind), *table, kp, vp, kp.stride(0), *outs)
    q = W.normal_bf16_bits(rng, (3, hk, d))
    attn = pka.BatchAttention()
    attn.plan(None, ptr, last, num_qo_heads=hk, num_kv_heads=hk, head_dim=d, page_size=16,
              layout="HND", kv_dtype=_name(group))
    o, lse = attn.run(bf16(q), kp, vp, i32(idx))
    torch.cuda.synchronize()
    assert (both[:, 1] == 0x5A).all() and pka.pka_get_device_error() == 0
    pools = [kv4.Pool.empty(pages, 16, hk, d, group, "HND", fill=0x5A) for _ in range(2)]
    for p, x, got, out in zip(pools, (k, v), (kp, vp), outs):
        p.data[:] = _appended(p, ref.bf16_bits_to_f64(x), ind, ptr, idx, last)
        assert np.array_equal(got.cpu().numpy(), p.data)
        rows = np.concatenate([kv4.request_rows(p, ptr, idx, r, int(m)) for r, m in enumerate(kv)])
        assert np.array_equal(f64(out), kv4.bf16_round(rows.astype(np.float32)).astype(float))
    _assert_decode(f64(o), f64(lse), kv4.attention(q, *pools, qo_indptr=np.arange(4),
                                                   kv_indptr=ptr, kv_indices=idx, kv_lens=kv,
                                                   hq=hk, hk=hk))


@pytest.mark.parametrize("hq,hk", [(8, 2), (8, 1)])
def test_many_short_requests(hq, hk):
    rng = np.random.default_rng(70)
    b = Batch(70, rng.integers(1, 6, 700), page=4, hq=hq, hk=hk, d=64, group=64)
    o, lse, info = b.run()
    assert info.num_decode_ctas <= 152
    _assert_decode(o, lse, b.want())


def test_captured_step_replayed():
    """Append, attention and read-back captured once and replayed over new rows: each
    replay's bytes and outputs are the eager calls'."""
    page, hq, hk, d = 16, 8, 2, 128
    rng = np.random.default_rng(80)
    params = pka.make_params(hq, hk, d, page, kv_dtype="int4_g32")
    size = pka.pka_kv_page_bytes(params)
    kv = np.array([50, 17])
    ptr, idx, last, pages = W.build_page_table(rng, kv, page, pool_pages=8)
    table = (i32(ptr), i32(idx), i32(last))
    ind, begin = i32([0, 1, 2]), i32(kv - 1)
    pools = torch.zeros(pages, 2, size, dtype=torch.uint8, device="cuda")
    q, o = (torch.zeros(2, hq, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lse = torch.zeros(2, hq, device="cuda")
    x, y, ko, vo = (torch.zeros(2, hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    attn = pka.BatchAttention()
    attn.plan(None, ptr, last, num_qo_heads=hq, num_kv_heads=hk, head_dim=d, page_size=page,
              kv_dtype="int4_g32")
    ids = i32(idx)

    def step(stream=None):
        k, v = pools[:, 0], pools[:, 1]
        pka.pka_append_paged_kv_cache(params, x, y, ind, *table, k, v, k.stride(0), stream=stream)
        attn.run(q, k, v, ids, out=o, lse=lse, stream=stream)
        pka.pka_read_paged_kv_cache(params, begin, ind, *table, k, v, k.stride(0), ko, vo,
                                    stream=stream)
    step()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step(stream)
    for i in range(3):
        for t, h in ((q, hq), (x, hk), (y, hk)):
            t.copy_(bf16(W.normal_bf16_bits(rng, (2, h, d))))
        pools.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (pools, o, lse, ko, vo)]
        pools.zero_()
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (pools, o, lse, ko, vo)):
            assert torch.equal(a, b)
        assert got[0].any() and pka.pka_get_device_error() == 0


# ---------------------------------------------------------------------------
# Pages of 4-bit pools
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("page,hk,d,group", [(1, 1, 128, 128), (4, 1, 64, 64), (16, 8, 128, 32),
                                             (5, 3, 128, 64), (64, 8, 128, 128), (3, 7, 64, 32)])
def test_copy_pages(layout, page, hk, d, group):
    """Whole pages and first slots, of one layer and of several, words with their codes."""
    rng = np.random.default_rng(page + hk)
    pages, layers, n = 23, 3, 7
    size = kv4.page_bytes(page, hk, d, group)
    data = rng.integers(0, 256, (layers, pages, 2, size), dtype=np.uint8)
    ids = rng.permutation(pages)
    src, dst = ids[:n], ids[n:2 * n]
    for slots in (None, rng.integers(0, page + 1, n)):
        kv = torch.from_numpy(data).cuda()
        pka.pka_copy_pages(pka.make_params(hk, hk, d, page, layout, kv_dtype=_name(group)),
                           kv[:, :, 0], kv[:, :, 1], i32(src), i32(dst),
                           None if slots is None else i32(slots))
        torch.cuda.synchronize()
        want = data.copy()
        code = page * hk * (d // 2)
        word = page * hk * (d // group) * 4
        for part, row in (((0, code), d // 2), ((code, code + word), d // group * 4)):
            shape = (page, hk, row) if layout == "NHD" else (hk, page, row)
            x = data[..., part[0]:part[1]].reshape(layers, pages, 2, *shape)
            y = x.copy()
            for i in range(n):
                k = page if slots is None else int(slots[i])
                if layout == "NHD":
                    y[:, dst[i], :, :k] = x[:, src[i], :, :k]
                else:
                    y[:, dst[i], :, :, :k] = x[:, src[i], :, :, :k]
            want[..., part[0]:part[1]] = y.reshape(layers, pages, 2, -1)
        got = kv.cpu().numpy()
        assert np.array_equal(got[..., :code + word], want[..., :code + word])
        assert np.array_equal(got[:, np.setdiff1d(np.arange(pages), dst)],
                              data[:, np.setdiff1d(np.arange(pages), dst)])


def test_a_step_with_everything_together():
    """A prompt quantised into the cache, forked into samples, extended by a rotating
    append, attended, and read back."""
    page, hq, hk, d, group = 16, 8, 2, 128, 64
    rng = np.random.default_rng(50)
    params = pka.make_params(hq, hk, d, page, kv_dtype=_name(group))
    size, pool_pages = pka.pka_kv_page_bytes(params), 64
    kv = torch.zeros(1, pool_pages, 2, size, dtype=torch.uint8, device="cuda")
    k, v = kv[0, :, 0], kv[0, :, 1]
    refs = torch.zeros(pool_pages, dtype=torch.int32, device="cuda")
    n = 41  # three pages, the last partly filled
    ptr, last = i32([0, 3]), i32([9])
    idx = torch.zeros(3, dtype=torch.int32, device="cuda")
    pka.pka_alloc_pages(refs, idx)
    rope = pka.make_rope(d)
    x = bf16(W.normal_bf16_bits(rng, (n, hk, d)))
    y = bf16(W.normal_bf16_bits(rng, (n, hk, d)))
    pka.pka_rope_append_paged_kv_cache(params, rope, None, None, x, y, i32([0, n]), ptr, idx, last,
                                       k, v, k.stride(0))
    # two samples
    child_ptr = i32([0, 3, 6])
    child_idx, src, dst, slots = (torch.full((m,), -1, dtype=torch.int32, device="cuda")
                                  for m in (6, 2, 2, 2))
    counts = torch.zeros(2, dtype=torch.int32, device="cuda")
    pka.pka_fork_pages(page, refs, ptr, idx, last, i32([0, 0]), child_ptr, child_idx, src, dst,
                       slots, counts)
    pka.pka_copy_pages(params, kv[:, :, 0], kv[:, :, 1], src, dst, slots, counts)
    # one more token each
    q = bf16(W.normal_bf16_bits(rng, (2, hq, d)))
    nk, nv = (bf16(W.normal_bf16_bits(rng, (2, hk, d))) for _ in range(2))
    q_out, clast = torch.empty_like(q), i32([10, 10])
    pka.pka_rope_append_paged_kv_cache(params, rope, q, q_out, nk, nv, i32([0, 1, 2]), child_ptr,
                                       child_idx, clast, k, v, k.stride(0))
    attn = pka.BatchAttention()
    attn.plan(None, np.array([0, 3, 6], np.int32), np.array([10, 10], np.int32), num_qo_heads=hq,
              num_kv_heads=hk, head_dim=d, page_size=page, kv_dtype=_name(group))
    o, lse = attn.run(q_out, k, v, child_idx)
    back = [torch.zeros(84, hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pka.pka_read_paged_kv_cache(params, None, i32([0, 42, 84]), child_ptr, child_idx, clast, k, v,
                                k.stride(0), *back)
    torch.cuda.synchronize()
    assert pka.pka_get_device_error() == 0
    kp, vp = (kv4.Pool(np.ascontiguousarray(t.cpu().numpy()), page, hk, d, group, "NHD")
              for t in (k, v))
    ci = child_idx.cpu().numpy()
    want = kv4.attention(bits_of(q_out), kp, vp, qo_indptr=np.arange(3), kv_indptr=[0, 3, 6],
                         kv_indices=ci, kv_lens=[42, 42], hq=hq, hk=hk)
    _assert_decode(f64(o), f64(lse), want)
    # V is what was appended, within half a step and the words' roundings
    vals = np.concatenate([f64(y), f64(nv[:1])])
    _, step, _ = kv4.quantize(vals.astype(np.float32), group)
    tol = np.repeat(step, group, -1) * (0.5 + 15 * 2.0 ** -8) + 2.0 ** -7 * (np.abs(vals) + 5)
    assert np.all(np.abs(f64(back[1][:42]) - vals) <= tol)
    assert torch.equal(back[0][:41], back[0][42:83])


@pytest.mark.parametrize("interleaved,rotary", [(False, 16), (False, 48), (True, 34)])
@pytest.mark.parametrize("d,group", SHAPES)
def test_rope_append_of_part_of_a_head(d, group, interleaved, rotary):
    """Half layouts whose pieces do not lie where a lane's codes do, and adjacent pairs of
    which a lane turns some."""
    test_rope_append(d, group, interleaved, rotary)


@pytest.mark.parametrize("rotary,interleaved", [(0, False), (32, False), (10, False), (0, True)])
@pytest.mark.parametrize("d,group", SHAPES)
def test_rope_append_layouts_agree(d, group, rotary, interleaved):
    """The same rows into NHD and HND pools read back as the same values; many rows, so that
    a warp takes several steps of one."""
    hq, hk, page, kv = 9, 5, 16, [700, 3, 1200]
    rng = np.random.default_rng(rotary + d)
    ptr, idx, last, pages = W.build_page_table(rng, np.asarray(kv), page)
    ind = i32(np.concatenate([[0], np.cumsum(kv)]))
    table = (i32(ptr), i32(idx), i32(last))
    n = sum(kv)
    q, k, v = (bf16(W.normal_bf16_bits(rng, (n, h, d))) for h in (hq, hk, hk))
    rope = pka.make_rope(rotary or d, interleaved=interleaved)
    q_outs, reads = [], []
    for layout in ("NHD", "HND"):
        params = pka.make_params(hq, hk, d, page, layout, kv_dtype=_name(group))
        pools = torch.zeros(pages, 2, pka.pka_kv_page_bytes(params), dtype=torch.uint8,
                            device="cuda")
        kp, vp = pools[:, 0], pools[:, 1]
        q_outs.append(torch.empty_like(q))
        pka.pka_rope_append_paged_kv_cache(params, rope, q, q_outs[-1], k, v, ind, *table, kp, vp,
                                           kp.stride(0))
        reads.append([torch.empty_like(k) for _ in range(2)])
        pka.pka_read_paged_kv_cache(params, None, ind, *table, kp, vp, kp.stride(0), *reads[-1])
    torch.cuda.synchronize()
    assert pka.pka_get_device_error() == 0 and torch.equal(*q_outs)
    for a, b in zip(*reads):
        assert torch.equal(a, b)
    # V is not rotated: off by half a step and the roundings of its words at most
    x = f64(v)
    _, step, _ = kv4.quantize(x.astype(np.float32), group)
    tol = np.repeat(step, group, -1) * (0.5 + 15 * 2.0 ** -8) + 2.0 ** -7 * (np.abs(x) + 5)
    assert np.all(np.abs(f64(reads[0][1]) - x) <= tol)
