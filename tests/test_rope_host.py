"""Rotary positions without a GPU: the frequencies that pka_rope_init makes,
what the entry points refuse before any device work, and pins of the oracle.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

import paged_kv_attention_plan_gb300 as pka
from oracle import cache
from paged_kv_attention_plan_gb300 import _pka

OK, INVALID, UNSUPPORTED = 0, 1, 3
A = 1 << 20  # an aligned address that a refused call never touches


def _turns(rope, n):
    t = np.array(rope.turns[:n], dtype=np.uint64).astype(np.int64)  # two's complement
    return t.astype(np.float64) / 2.0 ** 64


@pytest.mark.parametrize("kw", [
    dict(), dict(base=500000.0), dict(scaling="linear", factor=8.0),
    dict(base=500000.0, scaling="parts", factor=8.0, original_len=8192.0, low_rotations=1.0,
         high_rotations=4.0),
    dict(scaling="parts", factor=40.0, original_len=4096.0, low_rotations=1.0,
         high_rotations=32.0)])
@pytest.mark.parametrize("rotary", [2, 20, 64, 128])
def test_frequencies(rotary, kw):
    rope = pka.make_rope(rotary, **kw)
    want = cache.rope_frequencies(rotary, **kw) / (2 * math.pi)
    assert np.abs(_turns(rope, rotary // 2) - want).max() <= 2.0 ** -52
    assert rope.magnitude == 1.0 and rope.rotary_dim == rotary and rope.interleaved == 0


def test_own_frequencies_and_magnitude():
    f = np.array([0.0, 1.0, -1.0, math.pi])
    rope = pka.make_rope(8, frequencies=f, magnitude=1.25, interleaved=True)
    got = _turns(rope, 4)
    got[3] = abs(got[3])  # half a turn either way
    assert np.abs(got - f / (2 * math.pi)).max() <= 2.0 ** -52
    assert rope.magnitude == 1.25 and rope.interleaved == 1
    with pytest.raises(ValueError):
        pka.make_rope(8, frequencies=f[:3])


@pytest.mark.parametrize("kw,want", [
    (dict(rotary_dim=0), INVALID), (dict(rotary_dim=7), INVALID), (dict(rotary_dim=-2), INVALID),
    (dict(rotary_dim=130), UNSUPPORTED), (dict(base=0.5), INVALID),
    (dict(base=float("nan")), INVALID), (dict(base=float("inf")), INVALID),
    (dict(scaling=9), INVALID), (dict(scaling="linear", factor=0.5), INVALID),
    (dict(scaling="linear", factor=float("inf")), INVALID),
    (dict(scaling="parts", factor=2.0), INVALID),
    (dict(scaling="parts", factor=2.0, original_len=100.0, low_rotations=4.0,
          high_rotations=4.0), INVALID),
    (dict(magnitude=float("nan")), INVALID), (dict(magnitude=1e300), INVALID),
    (dict(frequencies=[3.2] * 32), INVALID), (dict(frequencies=[float("nan")] * 32), INVALID)])
def test_init_refusals(kw, want):
    with pytest.raises(pka.PkaError) as e:
        pka.make_rope(**{"rotary_dim": 64, **kw})
    assert e.value.status == want


def _apply(rope=None, transpose=0, dim=128, rows=4, pos=A, q=A, hq=8, qs=1024, qo=2 * A, qos=1024,
           k=3 * A, hk=2, ks=256, ko=4 * A, kos=256):
    rope = rope or pka.make_rope(64)
    return _pka.lib().pka_apply_rope(ctypes.byref(rope), transpose, dim, rows, pos, q, hq, qs, qo,
                                     qos, k, hk, ks, ko, kos, None)


@pytest.mark.parametrize("kw,want", [
    (dict(transpose=2), INVALID), (dict(dim=96), UNSUPPORTED), (dict(rows=-1), INVALID),
    (dict(hq=-1), INVALID), (dict(hk=1 << 20), UNSUPPORTED), (dict(pos=None), INVALID),
    (dict(q=None), INVALID), (dict(qo=None), INVALID), (dict(q=A + 8), INVALID),
    (dict(ko=A + 2), INVALID), (dict(qs=1016), INVALID), (dict(qs=1028), INVALID),
    (dict(kos=128), INVALID), (dict(qo=A, qos=2048), INVALID), (dict(rows=0), OK),
    (dict(hq=0, hk=0), OK)])
def test_apply_refusals(kw, want):
    assert _apply(**kw) == want


def test_apply_refuses_a_bad_rope():
    assert _apply(rope=pka.make_rope(128), dim=64, qs=512, qos=512, ks=128, kos=128) == INVALID
    assert _apply(rope=_pka.pka_rope()) == INVALID
    assert _pka.lib().pka_apply_rope(None, 0, 128, 1, A, A, 1, 128, A, 128, None, 0, 0, None, 0,
                                     None) == INVALID


def _append(params=None, rope=None, batch=2, nnz=4, q=A, qs=1024, qo=2 * A, kn=3 * A, ks=256,
            vn=4 * A, vs=256, pos=None, app=A, ptr=A, idx=A, last=A, k=5 * A, v=6 * A, stride=4096,
            pages=10):
    params = params or pka.make_params(8, 2, 128, 16)
    rope = rope or pka.make_rope(64)
    return _pka.lib().pka_rope_append_paged_kv_cache(
        ctypes.byref(params), ctypes.byref(rope), batch, nnz, q, qs, qo, kn, ks, vn, vs, pos, app,
        ptr, idx, last, k, v, stride, pages, None)


@pytest.mark.parametrize("kw,want", [
    (dict(batch=-1), INVALID), (dict(nnz=-1), INVALID), (dict(pages=-1), INVALID),
    (dict(q=None), INVALID), (dict(qo=None), INVALID), (dict(kn=None), INVALID),
    (dict(vn=None), INVALID), (dict(app=None), INVALID), (dict(ptr=None), INVALID),
    (dict(idx=None), INVALID), (dict(last=None), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(k=A + 8), INVALID), (dict(kn=A + 2), INVALID),
    (dict(stride=0), INVALID), (dict(stride=4097), INVALID), (dict(ks=255), INVALID),
    (dict(vs=128), INVALID), (dict(q=2 * A, qs=2048), INVALID), (dict(nnz=0), OK),
    (dict(batch=0), OK)])
def test_append_refusals(kw, want):
    assert _append(**kw) == want


def test_append_refuses_bad_params():
    p = lambda **kw: pka.make_params(**{**dict(num_qo_heads=8, num_kv_heads=2, head_dim=128,  # noqa
                                               page_size=16), **kw})
    assert _append(params=p(head_dim=96)) == UNSUPPORTED
    assert _append(params=p(kv_ragged=True)) == UNSUPPORTED
    assert _append(params=p(page_size=0)) == INVALID
    assert _append(params=p(layout=7)) == INVALID
    assert _append(params=p(kv_dtype="e4m3"), stride=4104) == INVALID
    assert _append(rope=pka.make_rope(128), params=p(head_dim=64), qs=512, ks=128,
                   vs=128) == INVALID


def test_binding_refuses_host_tensors(monkeypatch):
    """Tensors that are not on the GPU never reach the library."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    rope = pka.make_rope(64)
    x = torch.zeros(2, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        pka.pka_apply_rope(rope, torch.zeros(2, dtype=torch.int32), x, x)


# ---------------------------------------------------------------------------
# The oracle
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_is_complex_multiplication(interleaved):
    rng = np.random.default_rng(2)
    f = cache.rope_frequencies(12, base=100.0)
    x, pos = rng.standard_normal((5, 2, 16)), np.array([0, 1, 2, 50, 1000])
    y = cache.rope(x, pos, f, interleaved=interleaved, magnitude=1.5)
    for i in range(6):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 6)
        z = (x[:, :, a] + 1j * x[:, :, b]) * 1.5 * np.exp(1j * pos * f[i])[:, None]
        assert np.allclose(y[:, :, a], z.real, atol=1e-12)
        assert np.allclose(y[:, :, b], z.imag, atol=1e-12)
    assert np.array_equal(y[:, :, 12:], x[:, :, 12:])


def test_oracle_scores_depend_on_distance_alone():
    rng = np.random.default_rng(3)
    f = cache.rope_frequencies(16)
    q, k = rng.standard_normal((1, 1, 16)), rng.standard_normal((1, 1, 16))
    dots = [float(np.sum(cache.rope(q, [n + 7], f) * cache.rope(k, [n], f))) for n in (0, 5, 900)]
    assert np.allclose(dots, dots[0], atol=1e-9)


def test_oracle_transpose():
    rng = np.random.default_rng(4)
    f = cache.rope_frequencies(10)
    x, g, pos = rng.standard_normal((3, 2, 12)), rng.standard_normal((3, 2, 12)), [3, 0, 77]
    left = np.sum(cache.rope(x, pos, f, magnitude=1.3) * g)
    right = np.sum(x * cache.rope(g, pos, f, magnitude=1.3, transpose=True))
    assert abs(left - right) <= 1e-10
    back = cache.rope(cache.rope(x, pos, f), pos, f, transpose=True)
    assert np.abs(back - x).max() <= 1e-12


def test_binding_refuses_a_page_stride_that_is_not_the_pools(monkeypatch):
    """The pools know where their pages lie; another stride would reach past
    them.  (Checked on host tensors, with the library's entry replaced.)"""
    calls = []

    class Library:
        @staticmethod
        def pka_rope_append_paged_kv_cache(*args):
            calls.append(args)
            return 0

    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)  # host tensors' device
    monkeypatch.setattr(_pka, "lib", lambda: Library)
    rope, params = _pka.pka_rope(), pka.make_params(2, 2, 64, 4)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)  # noqa
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    both = torch.zeros(5, 2, 4, 2, 64, dtype=torch.bfloat16)  # K and V pages in turn

    def append(k, v, stride):
        return pka.pka_rope_append_paged_kv_cache(params, rope, None, None, x, x, i32(0, 1),
                                                  i32(0, 1), i32(0), i32(1), k, v, stride, stream=0)

    k, v = both[:, 0], both[:, 1]
    apart = k.contiguous(), v.contiguous()
    assert append(k, v, k.stride(0)) == 0 and append(*apart, apart[0].stride(0)) == 0
    assert append(k[:1], v[:1], 512) == 0  # one page: its stride leads nowhere
    assert len(calls) == 3
    for pools, stride in (((k, v), apart[0].stride(0)), (apart, k.stride(0)), ((k, v), 0)):
        with pytest.raises(ValueError, match="page_stride"):
            append(*pools, stride)
    assert len(calls) == 3


@pytest.mark.parametrize("off", [1, 2, 3])
def test_arrays_off_their_alignment_are_refused(off):
    """int32 arrays start at multiples of 4 bytes; the kernels could not read others."""
    assert _apply(pos=A + off) == INVALID
    for name in ("pos", "app", "ptr", "idx", "last"):
        assert _append(**{name: A + off}) == INVALID
