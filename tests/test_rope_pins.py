"""Rotary positions without a GPU: the oracle against closed forms, the
library's schedules (host code) against the oracle, and the refusals."""

import ctypes
import math

import numpy as np
import pytest

import paged_kv_cache_blk_gb300 as pkv
from oracle import rope as R
from paged_kv_cache_blk_gb300 import _binding as B

S = B.STATUS_CODES


@pytest.fixture(scope="module")
def lib():
    pkv.build()
    return pkv.load()


# ---- the oracle ---------------------------------------------------------------

@pytest.mark.parametrize("interleaved", [False, True])
def test_rotate_is_a_complex_product(interleaved):
    rng = np.random.default_rng(1)
    x = rng.normal(size=(5, 3, 16))
    pos = np.array([0, 1, 7, -4, 1000])
    f = R.inv_freq(8, 10000.0)
    y = R.rotate(x, pos, f, interleaved)
    a, b = (x[..., 0:8:2], x[..., 1:8:2]) if interleaved else (x[..., :4], x[..., 4:8])
    z = (a + 1j * b) * np.exp(1j * pos[:, None, None] * f)
    want = x.copy()
    if interleaved:
        want[..., 0:8:2], want[..., 1:8:2] = z.real, z.imag
    else:
        want[..., :4], want[..., 4:8] = z.real, z.imag
    assert np.allclose(y, want, atol=1e-12)
    assert np.array_equal(y[..., 8:], x[..., 8:]) and np.array_equal(y[0], x[0])


@pytest.mark.parametrize("interleaved", [False, True])
def test_scores_depend_on_the_distance_only(interleaved):
    rng = np.random.default_rng(2)
    q, k = rng.normal(size=(1, 1, 32)), rng.normal(size=(1, 1, 32))
    f = R.inv_freq(32, 500000.0)
    dot = lambda i, j: float((R.rotate(q, np.array([i]), f, interleaved)
                              * R.rotate(k, np.array([j]), f, interleaved)).sum())
    assert abs(dot(12, 5) - dot(907, 900)) < 1e-9
    assert abs(dot(12, 5) - dot(12, 6)) > 1e-3


def test_frequencies():
    f = R.inv_freq(4, 100.0)
    assert np.allclose(f, [1.0, 0.1], rtol=1e-15)
    assert np.allclose(R.inv_freq(4, 100.0, "linear", 8.0), f / 8)
    # the last pair of "base" scaling is stretched by the factor exactly, the first not at all
    g = R.inv_freq(64, 10000.0, "base", 4.0)
    h = R.inv_freq(64, 10000.0)
    assert math.isclose(g[0], h[0]) and math.isclose(g[-1], h[-1] / 4, rel_tol=1e-12)
    p = R.inv_freq(128, 10000.0, "by_parts", 16.0, 4096, 32, 1)
    h = R.inv_freq(128, 10000.0)
    turns = 4096 * h / (2 * math.pi)
    assert np.array_equal(p[turns >= 32], h[turns >= 32])
    assert np.array_equal(p[turns <= 1], h[turns <= 1] / 16)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and np.all(p[mid] < h[mid]) and np.all(p[mid] > h[mid] / 16)


def test_a_planted_mistake_shows():
    x = np.ones((1, 1, 4))
    f = R.inv_freq(4, 100.0)
    assert not np.allclose(R.rotate(x, np.array([3]), f, False), R.rotate(x, np.array([3]), f, True))
    assert not np.allclose(R.rotate(x, np.array([3]), f, False), R.rotate(x, np.array([-3]), f, False))


# ---- the library's schedules ----------------------------------------------------

@pytest.mark.parametrize("rd,base,kw", [
    (128, 10000.0, {}), (64, 500000.0, {}), (256, 1e6, {}), (2, 10000.0, {}),
    (128, 10000.0, dict(scaling="linear", factor=8.0)),
    (128, 10000.0, dict(scaling="base", factor=4.0)),
    (128, 500000.0, dict(scaling="by_parts", factor=16.0, original_len=8192)),
    (64, 10000.0, dict(scaling="by_parts", factor=4.0, original_len=2048, turns_fast=24,
                       turns_slow=2)),
])
def test_schedules(lib, rd, base, kw):
    r = pkv.Rope(rd, base=base, **kw)
    want = R.inv_freq(rd, base, **kw)
    got = np.array([r.struct.step[i] for i in range(rd // 2)], dtype=np.float64)
    # pow in 64 bits: a few units in the last place; and the step is a whole
    # number of 2^-64 turns, so half of that (2 pi 2^-65 radians) besides
    assert np.allclose(got * (2 * math.pi) / 2.0 ** 64, want, rtol=1e-14,
                       atol=2 * math.pi * 2.0 ** -65)
    assert math.isclose(r.attn_scale, R.attn_factor(kw.get("scaling"), kw.get("factor", 1.0)),
                        rel_tol=2 ** -24)
    assert all(r.struct.step[i] == 0 for i in range(rd // 2, 128))


def test_own_frequencies(lib):
    f = [1.0, 0.25, -0.5, 7.0, 0.0, 2 * math.pi, 1e-9, 100.0]
    r = pkv.Rope(16, inv_freq=f, attn_scale=1.25, interleaved=True)
    assert r.attn_scale == 1.25 and r.struct.interleaved == 1
    for i, x in enumerate(f):
        turn = x / (2 * math.pi)
        want = turn - math.floor(turn)
        got = r.struct.step[i] / 2.0 ** 64
        assert min(abs(got - want), 1 - abs(got - want)) < 1e-15 * max(1, abs(turn)) * 4


def test_schedule_refusals(lib):
    st = B._RopeStruct()
    p = ctypes.byref(st)
    ok = [128, 0, 1e4, 0, 1.0, 0.0, 32.0, 1.0]
    assert lib.pkv_rope_init(p, *ok) == S["PKV_OK"]
    for at, bad, want in [(0, 0, "INVALID_ARG"), (0, 7, "INVALID_ARG"), (0, -2, "INVALID_ARG"),
                          (0, 258, "UNSUPPORTED"), (1, 2, "INVALID_ARG"), (2, 0.0, "INVALID_ARG"),
                          (2, float("nan"), "INVALID_ARG"), (3, 4, "INVALID_ARG"),
                          (3, -1, "INVALID_ARG")]:
        a = list(ok)
        a[at] = bad
        assert lib.pkv_rope_init(p, *a) == S["PKV_ERR_" + want], (at, bad)
    for kind in (1, 2, 3):
        assert lib.pkv_rope_init(p, 128, 0, 1e4, kind, 0.5, 4096.0, 32.0, 1.0) \
            == S["PKV_ERR_INVALID_ARG"]
    assert lib.pkv_rope_init(p, 2, 0, 1e4, 2, 2.0, 0.0, 0.0, 0.0) == S["PKV_ERR_INVALID_ARG"]
    assert lib.pkv_rope_init(p, 128, 0, 1e4, 3, 2.0, 0.0, 32.0, 1.0) == S["PKV_ERR_INVALID_ARG"]
    assert lib.pkv_rope_init(p, 128, 0, 1e4, 3, 2.0, 4096.0, 1.0, 1.0) == S["PKV_ERR_INVALID_ARG"]
    assert lib.pkv_rope_init(None, *ok) == S["PKV_ERR_INVALID_ARG"]
    f = (ctypes.c_double * 4)(1, 1, float("inf"), 1)
    assert lib.pkv_rope_init_freqs(p, 8, 0, f, 1.0) == S["PKV_ERR_INVALID_ARG"]
    assert lib.pkv_rope_init_freqs(p, 4, 0, f, float("nan")) == S["PKV_ERR_INVALID_ARG"]
    assert lib.pkv_rope_init_freqs(p, 4, 0, None, 1.0) == S["PKV_ERR_INVALID_ARG"]
    with pytest.raises(ValueError):
        pkv.Rope(64, scaling="other")
    with pytest.raises(ValueError):
        pkv.Rope(64, inv_freq=[1.0] * 31)
    with pytest.raises(pkv.PkvError):
        pkv.Rope(63)


def _pool(**kw):
    base = dict(k_cache=16, v_cache=32, num_blocks=8, num_layers=2, block_size=16, num_kv_heads=2,
                head_dim=64, dtype=1)
    base.update(kw)
    return B._PoolStruct(*base.values())


def test_append_refusals(lib):
    p = ctypes.byref(_pool())

    def call(pool=p, rope=None, **kw):
        a = dict(layer=0, rope=rope or pkv.Rope(64).ref, bt=16, mb=4, offs=None, batch=2, seq=16,
                 pos=16, rpos=None, n=3, q=16, qs=256, hq=4, k=16, ks=128, v=16, vs=128, qo=16,
                 qos=256, sm=None, stream=None)
        a.update(kw)
        return lib.pkv_rope_append(pool, *a.values())

    bad, uns = S["PKV_ERR_INVALID_ARG"], S["PKV_ERR_UNSUPPORTED"]
    assert call(n=0) == S["PKV_OK"]
    for kw in (dict(layer=2), dict(layer=-1), dict(n=-1), dict(batch=-1), dict(hq=-1), dict(seq=0),
               dict(pos=0), dict(q=0), dict(qo=0), dict(k=0), dict(v=0), dict(bt=0), dict(mb=0),
               dict(q=24), dict(k=8), dict(v=24), dict(qo=8), dict(seq=6), dict(pos=6),
               dict(rpos=6), dict(bt=6), dict(sm=12), dict(qs=248), dict(qs=257), dict(ks=120),
               dict(vs=64), dict(qos=128), dict(ks=0), dict(ks=-128), dict(qs=1 << 61)):
        assert call(**kw) == bad, kw
    assert lib.pkv_rope_append(p, 0, None, 16, 4, None, 2, 16, 16, None, 3, 16, 256, 4, 16, 128, 16,
                               128, 16, 256, None, None) == bad
    assert call(rope=pkv.Rope(128).ref) == bad          # more than the head
    assert call(rope=pkv.Rope(20).ref) == uns           # not whole lanes
    assert call(rope=pkv.Rope(12, interleaved=True).ref) == uns
    assert call(pool=ctypes.byref(_pool(head_dim=96)), n=3) == uns
    assert call(pool=ctypes.byref(_pool(dtype=2, head_dim=96)), n=3) == uns
    assert call(pool=ctypes.byref(_pool(k_cache=0))) == bad
    zero = B._RopeStruct()
    assert call(rope=ctypes.byref(zero)) == bad
