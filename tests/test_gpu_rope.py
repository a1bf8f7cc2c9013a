"""GPU parity of pka_apply_rope and pka_rope_append_paged_kv_cache against the
float64 oracle.

Tolerances.  A rotated element is y = m (a c -+ b s) in float32, rounded once:
the sine and cosine are off by at most 2^-22 (angle 2^-23.3, function 2^-23),
the product with m, the two products and the sum add 4 half steps of 2^-24, so
|error| <= 2^-20 m (|a| + |b|) before the last rounding, which adds half a step
of the type: 2^-8 |y| (bf16), or 2^-4 |y| and at least half the smallest
subnormal, 2^-10 (e4m3, in units of the scale).  Elements that are not rotated
keep their bits.  The angle itself, n f, carries the 64-bit roundings of both
sides: the oracle's product, 2 pi, the quotient by it (half a step of 2^-52
each) and two powers (a whole step each): at most 8 * 2^-53 |n f|.
"""
import math

import numpy as np
import pytest
import torch

import paged_kv_attention_plan_gb300 as pka
from inputs import workloads as W
from oracle import cache, ref
from tests.gpu_util import bf16, bits_of, i32

pytestmark = pytest.mark.gpu

ARITH, BF16_HALF, E4M3_HALF, E4M3_TINY = 2.0 ** -20, 2.0 ** -8, 2.0 ** -4, 2.0 ** -10
FAR = 8 * 2.0 ** -53

SCALING = {
    "none": dict(base=10000.0),
    "linear": dict(base=10000.0, scaling="linear", factor=4.0),
    "parts": dict(base=500000.0, scaling="parts", factor=8.0, original_len=8192.0,
                  low_rotations=1.0, high_rotations=4.0),
}


def _rope(rotary, interleaved=False, scaling="none", magnitude=1.0):
    return (pka.make_rope(rotary, interleaved=interleaved, magnitude=magnitude, **SCALING[scaling]),
            cache.rope_frequencies(rotary, **SCALING[scaling]))


def _bound(x, want, freqs, interleaved, magnitude, positions):
    """The arithmetic's part of the tolerance, element by element."""
    rd = 2 * len(freqs)
    i = np.arange(rd // 2)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + rd // 2)
    size = np.zeros_like(want)
    both = np.abs(x[:, :, first]) + np.abs(x[:, :, second])
    turned = FAR * np.abs(np.asarray(positions, np.float64))[:, None, None] * np.abs(freqs)
    size[:, :, first] = size[:, :, second] = both * (ARITH + turned)
    return abs(magnitude) * size


def _assert_rotated(got_bits, x_bits, positions, freqs, *, interleaved, magnitude=1.0,
                    transpose=False):
    x = ref.bf16_bits_to_f64(x_bits)
    want = cache.rope(x, positions, freqs, interleaved=interleaved, magnitude=magnitude,
                      transpose=transpose)
    got = ref.bf16_bits_to_f64(got_bits)
    tol = _bound(x, want, freqs, interleaved, magnitude, positions) * (1 + BF16_HALF)
    assert np.all(np.abs(got - want) <= tol + BF16_HALF * np.abs(want))
    rd = 2 * len(freqs)
    assert np.array_equal(got_bits[:, :, rd:], x_bits[:, :, rd:])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rotary", [(64, 64), (64, 32), (64, 16), (64, 2), (64, 40), (64, 62),
                                      (128, 128), (128, 64), (128, 16), (128, 48), (128, 96),
                                      (128, 4), (128, 24), (128, 126)])
def test_layouts_and_parts_of_the_head(d, rotary, interleaved):
    rng = np.random.default_rng(rotary + d)
    rows, hq, hk = 37, 5, 3
    q, k = W.normal_bf16_bits(rng, (rows, hq, d)), W.normal_bf16_bits(rng, (rows, hk, d))
    pos = rng.integers(0, 5000, rows).astype(np.int32)
    rope, freqs = _rope(rotary, interleaved)
    qd, kd = bf16(q), bf16(k)
    qo, ko = torch.full_like(qd, float("nan")), torch.full_like(kd, float("nan"))
    pka.pka_apply_rope(rope, i32(pos), qd, qo, kd, ko)
    torch.cuda.synchronize()
    _assert_rotated(bits_of(qo), q, pos, freqs, interleaved=interleaved)
    _assert_rotated(bits_of(ko), k, pos, freqs, interleaved=interleaved)
    assert np.array_equal(bits_of(qd), q) and np.array_equal(bits_of(kd), k)


@pytest.mark.parametrize("rows,hq,hk", [(1, 1, 1), (1, 32, 8), (3, 64, 1), (8, 7, 0), (9, 0, 9),
                                        (700, 32, 8), (5000, 8, 2)])
def test_row_and_head_counts(rows, hq, hk):
    """One token to thousands, few heads and many, q or k alone."""
    rng = np.random.default_rng(rows)
    d = 128
    pos = rng.integers(0, 100000, rows).astype(np.int32)
    rope, freqs = _rope(d)
    q = W.normal_bf16_bits(rng, (rows, hq, d)) if hq else None
    k = W.normal_bf16_bits(rng, (rows, hk, d)) if hk else None
    qd, kd = (None if x is None else bf16(x) for x in (q, k))
    qo, ko = (None if x is None else torch.empty_like(x) for x in (qd, kd))
    pka.pka_apply_rope(rope, i32(pos), qd, qo, kd, ko)
    torch.cuda.synchronize()
    for x, y in ((q, qo), (k, ko)):
        if x is not None:
            _assert_rotated(bits_of(y), x, pos, freqs, interleaved=False)


def test_no_rows():
    """Calls without rows, or without requests, do nothing."""
    rope, _ = _rope(64)
    q, pos = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda"), i32([])
    pka.pka_apply_rope(rope, pos, q, q, q, q)
    params = pka.make_params(4, 4, 64, 4)
    pool = torch.zeros(3, 4, 4, 64, dtype=torch.bfloat16, device="cuda")
    table = [i32(x) for x in ([0, 0], [0, 1], [2], [3])]
    pka.pka_rope_append_paged_kv_cache(params, rope, q, q, q, q, *table, pool, pool, pool.stride(0))
    one = torch.ones(1, 4, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(one)
    for t in (table, [i32(x) for x in ([0], [0], [], [])]):  # a padded row of no request
        pka.pka_rope_append_paged_kv_cache(params, rope, one, out, one, one, *t, pool, pool,
                                           pool.stride(0))
    torch.cuda.synchronize()
    assert not pool.any() and not out.any() and pka.pka_get_device_error() == 0


@pytest.mark.parametrize("scaling", ["none", "linear", "parts"])
def test_far_positions_and_scaling(scaling):
    """Angles of positions up to the largest int32, and of negative ones."""
    rng = np.random.default_rng(5)
    pos = np.array([0, 1, -1, 4095, 131071, 1 << 20, (1 << 24) + 1, (1 << 30) + 12345,
                    (1 << 31) - 1, -(1 << 31)], np.int32)
    q = W.normal_bf16_bits(rng, (len(pos), 4, 128))
    rope, freqs = _rope(128, scaling=scaling, magnitude=1.2)
    qd = bf16(q)
    qo = torch.empty_like(qd)
    pka.pka_apply_rope(rope, i32(pos), qd, qo)
    torch.cuda.synchronize()
    _assert_rotated(bits_of(qo), q, pos, freqs, interleaved=False, magnitude=1.2)


def test_own_frequencies():
    rng = np.random.default_rng(6)
    f = np.concatenate([[0.0, math.pi, -1.0], rng.uniform(-3, 3, 29)])
    pos = rng.integers(-1000, 1000, 11).astype(np.int32)
    q = W.normal_bf16_bits(rng, (11, 2, 64))
    rope = pka.make_rope(64, frequencies=f, interleaved=True)
    qd = bf16(q)
    pka.pka_apply_rope(rope, i32(pos), qd, qd)
    torch.cuda.synchronize()
    _assert_rotated(bits_of(qd), q, pos, f, interleaved=True)


@pytest.mark.parametrize("interleaved,rotary", [(False, 128), (True, 128), (False, 64),
                                                (True, 32), (False, 20)])
def test_slices_of_a_fused_row_and_in_place(interleaved, rotary):
    """q and k as slices of one projection's rows, rotated where they lie; the
    v part of the rows keeps its bits."""
    rng = np.random.default_rng(rotary)
    rows, hq, hk, d = 65, 6, 2, 128
    x = W.normal_bf16_bits(rng, (rows, hq + 2 * hk, d))
    pos = rng.integers(0, 9000, rows).astype(np.int32)
    rope, freqs = _rope(rotary, interleaved)
    xd = bf16(x)
    q, k = xd[:, :hq], xd[:, hq:hq + hk]
    qo, ko = torch.empty(rows, hq, d, dtype=q.dtype, device="cuda"), torch.empty(
        rows, hk, d, dtype=q.dtype, device="cuda")
    pka.pka_apply_rope(rope, i32(pos), q, qo, k, ko)
    pka.pka_apply_rope(rope, i32(pos), q, q, k, k)
    torch.cuda.synchronize()
    got = bits_of(xd)
    _assert_rotated(got[:, :hq], x[:, :hq], pos, freqs, interleaved=interleaved)
    assert np.array_equal(bits_of(qo), got[:, :hq])
    assert np.array_equal(bits_of(ko), got[:, hq:hq + hk])
    assert np.array_equal(got[:, hq + hk:], x[:, hq + hk:])


@pytest.mark.parametrize("interleaved,rotary,d", [(False, 128, 128), (True, 64, 128),
                                                  (False, 36, 64)])
def test_transpose_is_the_gradient(interleaved, rotary, d):
    """The transposed map against the formula, and against differences of the
    forward map: for L = <R x, g>, dL/dx_e = (L(x + h e) - L(x - h e)) / 2h."""
    rng = np.random.default_rng(rotary)
    rows = 5
    g = W.normal_bf16_bits(rng, (rows, 2, d))
    pos = rng.integers(0, 3000, rows).astype(np.int32)
    rope, freqs = _rope(rotary, interleaved, magnitude=1.1)
    gd = bf16(g)
    dx = torch.empty_like(gd)
    pka.pka_apply_rope(rope, i32(pos), gd, dx, transpose=True)
    torch.cuda.synchronize()
    _assert_rotated(bits_of(dx), g, pos, freqs, interleaved=interleaved, magnitude=1.1,
                    transpose=True)
    gv, got = ref.bf16_bits_to_f64(g), ref.bf16_bits_to_f64(bits_of(dx))
    x = rng.standard_normal((rows, 2, d))
    h = 1e-3

    def loss(z):
        return float(np.sum(cache.rope(z, pos, freqs, interleaved=interleaved, magnitude=1.1) * gv))

    for _ in range(24):
        e = tuple(rng.integers(0, n) for n in x.shape)
        up, down = x.copy(), x.copy()
        up[e] += h
        down[e] -= h
        want = (loss(up) - loss(down)) / (2 * h)
        # the map is linear, so the difference is exact up to float64 rounding of the sums
        tol = BF16_HALF * abs(want) + ARITH * 1.1 * 2 * np.abs(gv).max() + 1e-9
        assert abs(got[e] - want) <= tol


def test_nan_and_infinity_stay_in_their_pair():
    """A NaN or an infinity reaches its own pair and nothing else, and elements
    past rotary_dim keep their bits, NaN payloads among them."""
    rng = np.random.default_rng(9)
    for interleaved in (False, True):
        q = W.normal_bf16_bits(rng, (3, 2, 64))
        q[0, 0, 3] = 0x7F80  # inf
        q[1, 1, 5] = 0x7FC1  # NaN
        q[2, 0, 40] = 0xFFC5  # NaN past the rotated part
        q[2, 1, 63] = 0xFF80
        rope, _ = _rope(32, interleaved)
        pos = np.array([7, 0, 11], np.int32)
        qd = bf16(q)
        qo = torch.empty_like(qd)
        pka.pka_apply_rope(rope, i32(pos), qd, qo)
        torch.cuda.synchronize()
        got = bits_of(qo)
        bad = ~np.isfinite(ref.bf16_bits_to_f64(got))
        pairs = [(0, 0, 2), (0, 0, 3), (1, 1, 4), (1, 1, 5)] if interleaved else \
            [(0, 0, 3), (0, 0, 19), (1, 1, 5), (1, 1, 21)]
        want = np.zeros_like(bad)
        for p in pairs + [(2, 0, 40), (2, 1, 63)]:
            want[p] = True
        assert np.array_equal(bad, want)
        assert np.array_equal(got[:, :, 32:], q[:, :, 32:])


# ---------------------------------------------------------------------------
# The append that rotates
# ---------------------------------------------------------------------------

def _check_append(b, rope_kw, rotary, *, scales=(1.0, 1.0), with_q=True, positions=None, pad=0,
                  magnitude=1.0, interleaved=False):
    rope, freqs = _rope(rotary, interleaved, magnitude=magnitude, **rope_kw)
    f8 = b.kv_dtype == "e4m3"
    params = pka.make_params(b.num_qo_heads, b.num_kv_heads, b.head_dim, b.page_size, b.layout,
                             kv_dtype=b.kv_dtype, k_scale=scales[0], v_scale=scales[1])
    rows = b.nnz_q
    grow = lambda x: np.concatenate([x, np.full((pad,) + x.shape[1:], 0x7FC1, np.uint16)])  # noqa
    to = (lambda x: torch.from_numpy(x.copy()).cuda()) if f8 else bf16
    k, v = to(b.k_pool), to(b.v_pool)
    q = bf16(grow(b.q))
    q_out = torch.full_like(q, 3.0)
    pos_d = None if positions is None else i32(positions)
    pka.pka_rope_append_paged_kv_cache(
        params, rope, q if with_q else None, q_out if with_q else None, bf16(grow(b.k_new)),
        bf16(grow(b.v_new)), i32(b.qo_indptr), i32(b.kv_indptr), i32(b.kv_indices),
        i32(b.last_page_len), k, v, k.stride(0), positions=pos_d)
    torch.cuda.synchronize()
    assert pka.pka_get_device_error() == 0
    where = cache.append_slots(b.qo_indptr, b.kv_indptr, b.kv_indices, b.last_page_len,
                               b.page_size)
    pos = np.array([w[1] for w in where]) if positions is None else np.asarray(positions)[:rows]
    if with_q:
        got = bits_of(q_out)
        _assert_rotated(got[:rows], b.q, pos, freqs, interleaved=interleaved, magnitude=magnitude)
        assert np.all(got[rows:] == 0x4040)  # rows of no request stay as they were
    # V, and every slot that no row was appended to, bit for bit
    k_ref, v_ref = ref.append_paged_kv_cache(
        b.k_new, b.v_new, b.qo_indptr, b.k_pool, b.v_pool, kv_indptr=b.kv_indptr,
        kv_indices=b.kv_indices, last_page_len=b.last_page_len, page_size=b.page_size,
        layout=b.layout, kv_dtype=b.kv_dtype, k_scale=scales[0], v_scale=scales[1])
    host = (lambda t: t.cpu().numpy()) if f8 else bits_of
    got_k, got_v = host(k), host(v)
    assert np.array_equal(got_v, v_ref)
    page, slot = np.array([w[2] for w in where], int), np.array([w[3] for w in where], int)
    swap = (lambda x: x) if b.layout == "NHD" else (lambda x: x.transpose(0, 2, 1, 3))
    new = swap(got_k)[page, slot].copy()
    rest, rest_ref = swap(got_k).copy(), swap(k_ref).copy()
    rest[page, slot] = rest_ref[page, slot] = 0
    assert np.array_equal(rest, rest_ref)
    if not f8:
        _assert_rotated(new, b.k_new, pos, freqs, interleaved=interleaved, magnitude=magnitude)
        return
    x = ref.bf16_bits_to_f64(b.k_new)
    want = cache.rope(x, pos, freqs, interleaved=interleaved, magnitude=magnitude) / scales[0]
    got = ref.e4m3_to_f64(new)
    tol = _bound(x, want, freqs, interleaved, magnitude, pos) / scales[0] * (1 + E4M3_HALF)
    tol = tol + 2.0 ** -24 * np.abs(want)  # the division
    want = np.clip(want, -448.0, 448.0)
    assert np.all(np.abs(got - want) <= tol + np.maximum(E4M3_HALF * np.abs(want), E4M3_TINY))


def _batch(seed, page_size, layout, d, kv_dtype="bf16", hq=8, hk=2):
    b = W.make_paged_batch(seed, [3, 1, 0, 17, 40, 1], [6, 2, 5, 40, 41, 1], page_size=page_size,
                           layout=layout, hq=hq, hk=hk, d=d, append_new=True)
    if kv_dtype == "e4m3":
        rng = np.random.default_rng(seed)
        b.kv_dtype = "e4m3"
        b.k_pool, b.v_pool = (W.e4m3_codes(rng, b.k_pool.shape) for _ in range(2))
    return b


@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("page_size", [1, 4, 16])
@pytest.mark.parametrize("d,rotary,interleaved", [(64, 64, False), (128, 64, True),
                                                  (128, 128, False), (64, 22, False)])
def test_append_rotated(layout, page_size, d, rotary, interleaved):
    _check_append(_batch(page_size, page_size, layout, d), {}, rotary, interleaved=interleaved)


@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("page_size,d,rotary,interleaved,scales", [
    (1, 64, 64, False, (1.0, 1.0)), (4, 128, 128, False, (0.3, 2.5)),
    (16, 128, 32, True, (0.004, 0.75)), (16, 128, 20, False, (0.25, 0.02))])
def test_append_rotated_e4m3(layout, page_size, d, rotary, interleaved, scales):
    """k_scale 0.004 drives most values past 448."""
    _check_append(_batch(page_size + 7, page_size, layout, d, "e4m3"), {}, rotary, scales=scales,
                  interleaved=interleaved)


@pytest.mark.parametrize("scale", [1.0, 0.3, 0.004, 2.5, 1.0 / 3.0, 7.0, 1e-3, 0.02, 448.0, 1e-20,
                                   1e-17, 3e30])
def test_append_e4m3_codes_of_every_bf16_value(scale):
    """V of every bit pattern, divided by the scale and rounded: the codes that
    pka_append_paged_kv_cache stores, infinities and NaN among them."""
    v = np.arange(1 << 16, dtype=np.uint16).reshape(256, 2, 128)
    k = np.zeros_like(v)
    params = pka.make_params(8, 2, 128, 16, kv_dtype="e4m3", v_scale=scale)
    pools = [torch.zeros(16, 16, 2, 128, dtype=torch.uint8, device="cuda") for _ in range(4)]
    table = [i32(x) for x in ([0, 256], [0, 16], np.arange(16), [16])]
    pka.pka_rope_append_paged_kv_cache(params, _rope(128)[0], None, None, bf16(k), bf16(v), *table,
                                       pools[0], pools[1], pools[0].stride(0))
    pka.pka_append_paged_kv_cache(params, bf16(k), bf16(v), *table, pools[2], pools[3],
                                  pools[2].stride(0))
    torch.cuda.synchronize()
    got = pools[1].cpu().numpy().reshape(v.shape)
    assert np.array_equal(got, pools[3].cpu().numpy().reshape(v.shape))
    with np.errstate(all="ignore"):
        finite = np.isfinite(ref.bf16_bits_to_f64(v))
        want = ref.quantize_kv_e4m3(v, scale)
    assert np.array_equal(got[finite], want[finite])


def test_append_padded_batch_and_given_positions():
    b = _batch(3, 4, "NHD", 128)
    _check_append(b, dict(scaling="parts"), 128, pad=21, magnitude=1.2)
    rng = np.random.default_rng(1)
    pos = rng.integers(0, 1 << 20, b.nnz_q).astype(np.int32)
    _check_append(b, {}, 128, positions=pos)
    _check_append(b, {}, 128, with_q=False)


def test_append_many_requests():
    """More requests than one round of the row search, empty ones among them."""
    rng = np.random.default_rng(8)
    new = rng.integers(0, 3, 1500)
    b = W.make_paged_batch(8, new, new + rng.integers(1, 9, 1500), page_size=4, hq=2, hk=1, d=64,
                           append_new=True)
    _check_append(b, {}, 64)


def test_append_slices_of_a_fused_row_with_5d_pools():
    rng = np.random.default_rng(12)
    b = _batch(12, 4, "NHD", 128)
    x = W.normal_bf16_bits(rng, (b.nnz_q, 8 + 4, 128))
    b.q, b.k_new, b.v_new = (np.ascontiguousarray(x[:, s]) for s in
                             (slice(0, 8), slice(8, 10), slice(10, 12)))
    xd = bf16(x)
    rope, freqs = _rope(128)
    params = pka.make_params(8, 2, 128, 4)
    pool = torch.stack([bf16(b.k_pool), bf16(b.v_pool)], dim=1).contiguous()
    q_out = torch.empty(b.nnz_q, 8, 128, dtype=torch.bfloat16, device="cuda")
    k, v = pool[:, 0], pool[:, 1]
    pka.pka_rope_append_paged_kv_cache(params, rope, xd[:, :8], q_out, xd[:, 8:10], xd[:, 10:],
                                       i32(b.qo_indptr), i32(b.kv_indptr), i32(b.kv_indices),
                                       i32(b.last_page_len), k, v, k.stride(0))
    torch.cuda.synchronize()
    where = cache.append_slots(b.qo_indptr, b.kv_indptr, b.kv_indices, b.last_page_len, 4)
    pos = np.array([w[1] for w in where])
    page, slot = np.array([w[2] for w in where]), np.array([w[3] for w in where])
    _assert_rotated(bits_of(q_out), b.q, pos, freqs, interleaved=False)
    _assert_rotated(bits_of(k)[page, slot], b.k_new, pos, freqs, interleaved=False)
    assert np.array_equal(bits_of(v)[page, slot], b.v_new)


def test_append_bad_page_is_skipped_and_noted():
    b = _batch(4, 4, "NHD", 64)
    idx = b.kv_indices.copy()
    r = 4  # 41 keys, 40 new: its pages 1 and 2 hold new rows only
    first = int(b.kv_indptr[r])
    idx[first + 1], idx[first + 2] = -7, b.k_pool.shape[0]
    params = pka.make_params(8, 2, 64, 4)
    rope, _ = _rope(64)
    k, v = bf16(b.k_pool), bf16(b.v_pool)
    pka.pka_rope_append_paged_kv_cache(params, rope, None, None, bf16(b.k_new), bf16(b.v_new),
                                       i32(b.qo_indptr), i32(b.kv_indptr), i32(idx),
                                       i32(b.last_page_len), k, v, k.stride(0))
    torch.cuda.synchronize()
    assert pka.pka_get_device_error() == 2  # PKA_ERR_METADATA
    assert pka.pka_get_device_error() == 0
    good = bf16(b.v_pool)
    pka.pka_append_paged_kv_cache(params, bf16(b.k_new), bf16(b.v_new), i32(b.qo_indptr),
                                  i32(b.kv_indptr), i32(b.kv_indices), i32(b.last_page_len),
                                  torch.empty_like(good), good, k.stride(0))
    skipped = b.kv_indices[[first + 1, first + 2]]
    want = bits_of(good)
    want[skipped] = b.v_pool[skipped]
    assert np.array_equal(bits_of(v), want)


def test_rotate_append_attend():
    """The serving step as it is used: rotate and append, then attend."""
    from tests.gpu_util import assert_parity, f64
    b = W.make_paged_batch(21, [1, 40, 1, 7], [300, 90, 17, 7], page_size=16, hq=32, hk=8, d=128,
                           append_new=True)
    rope, freqs = _rope(128, scaling="parts")
    params = pka.make_params(32, 8, 128, 16)
    k, v, q = bf16(b.k_pool), bf16(b.v_pool), bf16(b.q)
    idx = i32(b.kv_indices)
    pka.pka_rope_append_paged_kv_cache(params, rope, q, q, bf16(b.k_new), bf16(b.v_new),
                                       i32(b.qo_indptr), i32(b.kv_indptr), idx,
                                       i32(b.last_page_len), k, v, k.stride(0))
    attn = pka.BatchAttention()
    attn.plan(b.qo_indptr, b.kv_indptr, b.last_page_len, num_qo_heads=32, num_kv_heads=8,
              head_dim=128, page_size=16)
    o, lse = attn.run(q, k, v, idx)
    torch.cuda.synchronize()
    # the oracle attends over the rotated rows that the call stored
    where = cache.append_slots(b.qo_indptr, b.kv_indptr, b.kv_indices, b.last_page_len, 16)
    pos = np.array([w[1] for w in where])
    _assert_rotated(bits_of(q), b.q, pos, freqs, interleaved=False)
    o_ref, lse_ref = ref.batch_attention(
        bits_of(q), bits_of(k), bits_of(v), qo_indptr=b.qo_indptr, kv_indptr=b.kv_indptr,
        kv_indices=b.kv_indices, last_page_len=b.last_page_len, page_size=16, num_qo_heads=32,
        num_kv_heads=8)
    assert_parity(f64(o), f64(lse), o_ref, lse_ref)


def test_captured_on_another_stream_and_replayed():
    """A captured append (first call of its kind inside the capture) replayed
    with new rows and another page table, on a stream of its own."""
    b = _batch(31, 4, "HND", 128)
    params = pka.make_params(8, 2, 128, 4, "HND")
    rope, freqs = _rope(128, True)
    k, v, kn, vn = bf16(b.k_pool), bf16(b.v_pool), bf16(b.k_new), bf16(b.v_new)
    q = bf16(b.q)
    q_out = torch.empty_like(q)
    app, ptr, idx, last = (i32(x) for x in (b.qo_indptr, b.kv_indptr, b.kv_indices,
                                            b.last_page_len))
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        pka.pka_rope_append_paged_kv_cache(params, rope, q, q_out, kn, vn, app, ptr, idx, last, k,
                                           v, k.stride(0), stream=stream)
    for seed in (1, 2):
        rng = np.random.default_rng(seed)
        b.k_new, b.v_new = (W.normal_bf16_bits(rng, b.k_new.shape) for _ in range(2))
        b.kv_indices = rng.permutation(b.k_pool.shape[0])[:len(b.kv_indices)].astype(np.int32)
        for t, x in ((kn, bf16(b.k_new)), (vn, bf16(b.v_new)), (idx, i32(b.kv_indices)),
                     (k, bf16(b.k_pool)), (v, bf16(b.v_pool))):
            t.copy_(x)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        where = cache.append_slots(b.qo_indptr, b.kv_indptr, b.kv_indices, b.last_page_len, 4)
        pos = np.array([w[1] for w in where])
        page, slot = np.array([w[2] for w in where]), np.array([w[3] for w in where])
        _assert_rotated(bits_of(k)[page, :, slot], b.k_new, pos, freqs, interleaved=True)
        assert np.array_equal(bits_of(v)[page, :, slot], b.v_new)
        _assert_rotated(bits_of(q_out), b.q, pos, freqs, interleaved=True)


@pytest.mark.parametrize("exponent", [-149, -140, -128, -127, -126, 127])
def test_e4m3_codes_of_scales_at_the_ends_of_the_exponents(exponent):
    """Powers of two whose reciprocal is no float32, or barely one: zeros keep
    their code, every other value has that of its quotient."""
    scale = 2.0 ** exponent
    v = np.arange(1 << 16, dtype=np.uint16).reshape(256, 2, 128)
    params = pka.make_params(8, 2, 128, 16, kv_dtype="e4m3", k_scale=scale, v_scale=scale)
    pools = [torch.zeros(16, 16, 2, 128, dtype=torch.uint8, device="cuda") for _ in range(4)]
    table = [i32(x) for x in ([0, 256], [0, 16], np.arange(16), [16])]
    pka.pka_rope_append_paged_kv_cache(params, _rope(128)[0], None, None, bf16(v), bf16(v), *table,
                                       pools[0], pools[1], pools[0].stride(0),
                                       positions=i32(np.zeros(256)))
    pka.pka_append_paged_kv_cache(params, bf16(v), bf16(v), *table, pools[2], pools[3],
                                  pools[2].stride(0))
    torch.cuda.synchronize()
    got = [p.cpu().numpy().reshape(v.shape) for p in pools]
    with np.errstate(all="ignore"):
        x = ref.bf16_bits_to_f64(v)
        finite, want = np.isfinite(x), ref.quantize_kv_e4m3(v, scale)
    for codes in got[1:]:
        assert np.array_equal(codes[finite], want[finite])
    # K of position 0 is x c - y s with c = 1 and s = 0, where both of a pair are finite; a
    # zero may lose its sign
    pair = finite & np.roll(finite, 64, axis=2)
    assert np.array_equal(got[0][pair & (x != 0)], want[pair & (x != 0)])
    assert not np.any(got[0][pair & (x == 0)] & 0x7F)


@pytest.mark.parametrize("scale", [1.0, 0.25, 0.3, 0.02, 7.0])
@pytest.mark.parametrize("d,rotary,interleaved", [(128, 128, False), (128, 64, True),
                                                  (64, 20, False)])
def test_k_codes_of_position_0_are_the_plain_appends(d, rotary, interleaved, scale):
    """At position 0 the rotation is the identity, so K's codes are those of
    pka_append_paged_kv_cache, every finite bf16 value among them."""
    x = np.arange(1 << 16, dtype=np.uint16)
    x = x[(x & 0x7F80) != 0x7F80]
    x = np.resize(x, (len(x) // (2 * d) + 1) * 2 * d).reshape(-1, 2, d)
    rows = len(x)
    params = pka.make_params(2, 2, d, 16, kv_dtype="e4m3", k_scale=scale, v_scale=scale)
    pages = -(-rows // 16)
    pools = [torch.zeros(pages, 16, 2, d, dtype=torch.uint8, device="cuda") for _ in range(4)]
    table = [i32(a) for a in ([0, rows], [0, pages], np.arange(pages), [rows - 16 * (pages - 1)])]
    pka.pka_rope_append_paged_kv_cache(params, _rope(rotary, interleaved)[0], None, None, bf16(x),
                                       bf16(x), *table, pools[0], pools[1], pools[0].stride(0),
                                       positions=i32(np.zeros(rows)))
    pka.pka_append_paged_kv_cache(params, bf16(x), bf16(x), *table, pools[2], pools[3],
                                  pools[2].stride(0))
    torch.cuda.synchronize()
    got, want = (p.cpu().numpy().reshape(-1, 2, d)[:rows] for p in (pools[0], pools[2]))
    some = (x & 0x7FFF) != 0  # x c - y s of a negative zero may be a positive one
    assert np.array_equal(got[some], want[some]) and not np.any(got[~some] & 0x7F)
