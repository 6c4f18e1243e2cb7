"""Sparse decode without a GPU: the oracle against brute force and closed
forms, and the refusals of the three calls."""

import ctypes
import math

import numpy as np
import pytest

import paged_kv_cache_blk_gb300 as pkv
from oracle import sparse as SP
from oracle.oracle import attention_fp64
from paged_kv_cache_blk_gb300 import _binding as B

S = B.STATUS_CODES


@pytest.fixture(scope="module")
def lib():
    pkv.build()
    return pkv.load()


def test_exponent():
    assert SP.exponent(0.0) == -40 and SP.exponent(math.inf) == 40 and SP.exponent(math.nan) == 40
    for e in (-40, -7, 0, 5, 39):
        assert SP.exponent(127 * 2.0 ** e) == e
        assert SP.exponent(np.nextafter(127 * 2.0 ** e, np.inf)) == e + 1
    assert SP.exponent(1e30) == 40


def test_bounds_hold_every_key():
    rng = np.random.default_rng(1)
    for _ in range(20):
        rows = rng.normal(size=(16, 64)) * 10.0 ** rng.integers(-8, 8)
        codes, e = SP.block_bounds(rows)
        unit = 2.0 ** e
        assert np.all(codes[0] * unit >= rows.max(0)) and np.all(codes[1] * unit <= rows.min(0))
        assert np.all(codes[0] * unit < rows.max(0) + unit)
        assert np.abs(codes).max() > 63          # the unit is the smallest that fits


def test_scores_bound_the_logits_of_the_coded_query():
    rng = np.random.default_rng(2)
    q = rng.normal(size=(3, 32))
    blocks = rng.normal(size=(9, 8, 32))
    got = [SP.block_bounds(b) for b in blocks]
    s = SP.block_scores(q, np.array([c for c, _ in got]), [2.0 ** e for _, e in got])
    coded = np.array([c * 2.0 ** e for c, e in map(SP.query_codes, q)])
    assert np.max(np.abs(coded - q)) <= np.abs(q).max() / 63.5 / 2
    logits = np.einsum("gd,brd->bgr", coded, blocks).max((1, 2))
    assert np.all(s >= logits)


def test_selection():
    s = np.array([5.0, 1, 3, 3, 9, 3, 0, 2])
    assert SP.select(s, 8, 0, 0) == list(range(8)) and SP.select(s, 20, 1, 1) == list(range(8))
    assert SP.select(s, 3, 0, 0) == [0, 2, 4]            # of equal scores the lowest
    assert SP.select(s, 4, 0, 1) == [0, 2, 4, 7]
    assert SP.select(s, 4, 2, 2) == [0, 1, 6, 7]
    assert SP.select(-s, 2, 0, 0) == [1, 6]


def test_attention_over_all_entries_is_dense_attention():
    rng = np.random.default_rng(3)
    keys, values, q = rng.normal(size=(5, 4, 8)), rng.normal(size=(5, 4, 8)), rng.normal(size=(2, 8))
    out, mean, top = SP.sparse_attention(q, keys, values, [3, 0, 4, 1, 2], 4, 2, 14, 0.3)
    k, v = keys.reshape(20, 8)[2:17], values.reshape(20, 8)[2:17]
    want = np.stack([attention_fp64(x, k, v, 0.3) for x in q])
    assert np.allclose(out, want, atol=1e-12)
    assert np.all(mean >= np.abs(out) - 1e-12) and top.shape == (2,)
    none, _, _ = SP.sparse_attention(q, keys, values, [-1, 4], 4, 2, 9, 0.3)
    assert not none.any()


def test_planted_mistakes_show():
    rows = np.array([[1.0, -2.0], [0.3, 0.7]])
    codes, e = SP.block_bounds(rows)
    assert not np.array_equal(codes, np.rint(np.array([rows.max(0), rows.min(0)]) / 2.0 ** e))
    s = np.array([1.0, 1.0, 1.0])
    assert SP.select(s, 1, 0, 0) != [2]


# ---- refusals ---------------------------------------------------------------------

def _pool(**kw):
    base = dict(k_cache=16, v_cache=32, num_blocks=8, num_layers=2, block_size=16, num_kv_heads=2,
                head_dim=64, dtype=1)
    base.update(kw)
    return ctypes.byref(B._PoolStruct(*base.values()))


BAD, UNS = S["PKV_ERR_INVALID_ARG"], S["PKV_ERR_UNSUPPORTED"]


def test_update_refusals(lib):
    def call(pool=_pool(), **kw):
        a = dict(layer=0, bt=16, mb=4, lens=16, offs=None, first=None, batch=2, codes=16, scales=16,
                 stream=None)
        a.update(kw)
        return lib.pkv_update_block_bounds(pool, *a.values())

    assert call(batch=0) == S["PKV_OK"]
    for kw in (dict(layer=2), dict(layer=-1), dict(batch=-1), dict(bt=0), dict(mb=0), dict(lens=0),
               dict(codes=0), dict(scales=0), dict(codes=8), dict(scales=6), dict(bt=2),
               dict(lens=2), dict(offs=2), dict(first=2)):
        assert call(**kw) == BAD, kw
    assert call(pool=_pool(head_dim=32)) == UNS and call(pool=_pool(head_dim=96)) == UNS
    assert call(pool=_pool(dtype=9)) == UNS and call(pool=_pool(k_cache=0)) == BAD
    assert call(mb=1 << 28) == UNS


def test_select_refusals(lib):
    def call(pool=_pool(), **kw):
        a = dict(layer=0, codes=16, scales=16, q=16, hq=4, bt=16, mb=4, offs=None, batch=2, seq=16,
                 pos=16, n=3, k=8, sink=1, recent=1, sel=16, cnt=16, stream=None)
        a.update(kw)
        return lib.pkv_select_blocks(pool, *a.values())

    assert call(n=0) == S["PKV_OK"] and call(n=0, pool=_pool(k_cache=0, v_cache=0)) == S["PKV_OK"]
    for kw in (dict(layer=2), dict(batch=-1), dict(n=-1), dict(hq=0), dict(hq=3), dict(k=0),
               dict(sink=-1), dict(recent=-1), dict(sink=5, recent=4), dict(codes=0),
               dict(codes=4), dict(scales=0), dict(q=0), dict(q=8), dict(bt=0), dict(mb=0),
               dict(seq=0), dict(pos=0), dict(sel=0), dict(cnt=0), dict(sel=2), dict(cnt=2),
               dict(seq=2), dict(pos=2), dict(offs=2), dict(bt=2), dict(scales=2)):
        assert call(**kw) == BAD, kw
    assert call(hq=34) == UNS                     # 17 query heads a kv head
    assert call(pool=_pool(head_dim=256)) == UNS
    assert call(mb=400000) == UNS and call(mb=1 << 28) == UNS


def test_sparse_refusals(lib):
    def call(pool=_pool(), **kw):
        a = dict(layer=0, q=16, hq=4, scale=0.1, bt=16, mb=4, offs=None, batch=2, seq=16, pos=16,
                 n=3, sel=16, k=8, out=16, stream=None)
        a.update(kw)
        return lib.pkv_decode_attention_sparse(pool, *a.values())

    assert call(n=0) == S["PKV_OK"]
    for kw in (dict(layer=2), dict(batch=-1), dict(n=-1), dict(hq=0), dict(hq=3), dict(k=-1),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(q=0), dict(q=8),
               dict(out=0), dict(out=8), dict(bt=0), dict(mb=0), dict(seq=0), dict(pos=0),
               dict(sel=0), dict(sel=2), dict(bt=2), dict(seq=2), dict(pos=2), dict(offs=2)):
        assert call(**kw) == BAD, kw
    assert call(hq=34) == UNS
    assert call(pool=_pool(head_dim=96)) == UNS and call(pool=_pool(head_dim=256)) == UNS
    assert call(mb=1 << 28) == UNS
    assert call(pool=_pool(k_cache=0)) == BAD
