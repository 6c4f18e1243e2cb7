"""Windowed attention and tree verification without a GPU: the oracle against
closed forms, and what the C ABI refuses before it touches the device."""

import ctypes
import math

import numpy as np
import pytest

import paged_kv_cache_blk_gb300 as pkv
from oracle import masked as MK
from paged_kv_cache_blk_gb300 import _binding as B

S = B.STATUS_CODES
BAD, UNS, WS = S["PKV_ERR_INVALID_ARG"], S["PKV_ERR_UNSUPPORTED"], S["PKV_ERR_WORKSPACE"]


@pytest.fixture(scope="module")
def lib():
    pkv.build()
    return pkv.load()


# ---- the oracle -----------------------------------------------------------------

def test_window():
    assert MK.window_seen(5, 1, 0).tolist() == [0, 0, 0, 0, 0, 1]
    assert MK.window_seen(5, 2, 1).tolist() == [1, 0, 0, 0, 1, 1]
    assert MK.window_seen(5, 6, 0).all() and MK.window_seen(5, 0, 0).all()
    assert MK.window_seen(5, 1, 9).all() and MK.window_seen(0, 1, 0).tolist() == [1]
    for pos in range(12):  # a window moves with its query
        assert MK.window_seen(pos, 4, 0).sum() == min(4, pos + 1)


def test_tree():
    sees = np.array([[1, 0, 0], [1, 1, 0], [1, 0, 1]])
    assert MK.tree_seen(2, sees, 2, 3, 0, 0).tolist() == [1, 1, 1, 0, 1]
    assert MK.tree_seen(4, sees, 1, 5, 3, 1).tolist() == [1, 0, 0, 1, 1, 1, 0]
    assert MK.tree_seen(4, sees, 1, 0, 3, 0).tolist() == [0, 0, 1, 1, 1, 1, 0]  # position at least 4
    assert MK.tree_seen(0, np.zeros((1, 1)), 0, 0, 0, 0).tolist() == [0]
    # a chain's mask under no window is the causal mask
    n, ctx = 5, 3
    for i in range(n):
        assert np.array_equal(MK.tree_seen(ctx, np.tril(np.ones((n, n))), i, ctx + i, 0, 0),
                              np.arange(ctx + n) <= ctx + i)


def test_mask_words():
    sees = np.zeros((2, 70))
    sees[0, [0, 63]], sees[1, [64, 69]] = 1, 1
    assert MK.mask_words(sees, 2).tolist() == [[1 + 2 ** 63, 0], [0, 1 + 2 ** 5]]


def test_attention():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((2, 4)), rng.standard_normal((3, 4)), rng.standard_normal((3, 4))
    out, mean, top = MK.attention(q, k, v, np.array([0, 1, 0], bool), 0.5)  # one key: its value
    assert np.allclose(out, v[1]) and np.allclose(mean, np.abs(v[1]))
    assert top[0] == pytest.approx(np.abs(q[0] * k[1]).sum())
    assert not MK.attention(q, k, v, np.zeros(3, bool), 0.5)[0].any()       # none: zeros
    k[:] = k[0]
    assert np.allclose(MK.attention(q, k, v, np.ones(3, bool), 2.0)[0], v.mean(0))  # equal keys
    k = np.array([[1.0, 0, 0, 0], [0, 0, 0, 0], [9, 9, 9, 9]])
    got = MK.attention(np.array([[1.0, 0, 0, 0]]), k, v, np.array([1, 1, 0], bool), 1.0)[0]
    w = math.e / (1 + math.e)
    assert np.allclose(got, w * v[0] + (1 - w) * v[1])


def test_accept_moves():
    assert MK.accept_moves(10, [0, 2, 5]) == [(12, 11), (15, 12)]
    assert MK.accept_moves(10, [0, 1, 2]) == [] and MK.accept_moves(0, [3]) == [(3, 0)]


# ---- refusals of the C ABI --------------------------------------------------------

def _pool(**kw):
    base = dict(k_cache=16, v_cache=32, num_blocks=8, num_layers=2, block_size=16,
                num_kv_heads=2, head_dim=64, dtype=1)
    base.update(kw)
    return ctypes.byref(B._PoolStruct(*base.values()))


COMMON = [dict(layer=2), dict(layer=-1), dict(batch=-1), dict(hq=0), dict(hq=3),
          dict(scale=float("nan")), dict(scale=float("inf")), dict(q=0), dict(q=8), dict(out=0),
          dict(out=8), dict(bt=0), dict(bt=2), dict(mb=0), dict(lens=0), dict(lens=2),
          dict(offs=2), dict(sink=-1), dict(window=-1)]


def test_window_decode_refusals(lib):
    def call(pool=_pool(), **kw):
        a = dict(layer=0, q=16, hq=4, scale=0.1, bt=16, mb=4, lens=16, offs=None, batch=2,
                 window=8, sink=1, out=16, stream=None)
        a.update(kw)
        return lib.pkv_decode_attention_window(pool, *a.values())

    assert call(batch=0) == S["PKV_OK"]
    for kw in COMMON + [dict(window=0)]:
        assert call(**kw) == BAD, kw
    assert call(hq=34) == UNS and call(pool=_pool(head_dim=96)) == UNS
    assert call(mb=1 << 27) == UNS and call(pool=_pool(k_cache=0)) == BAD
    assert call(pool=_pool(dtype=9)) == UNS


CU = [dict(cu=0), dict(cu=4), dict(total=-1), dict(most=-1)]


def test_window_prefill_refusals(lib):
    def call(pool=_pool(), **kw):
        a = dict(layer=0, q=16, hq=4, scale=0.1, bt=16, mb=4, lens=16, offs=None, cu=16, batch=2,
                 total=6, most=4, window=8, sink=1, out=16, stream=None)
        a.update(kw)
        return lib.pkv_prefill_attention_window(pool, *a.values())

    for kw in (dict(batch=0), dict(total=0), dict(most=0)):
        assert call(**kw) == S["PKV_OK"]
    for kw in COMMON + CU + [dict(window=0)]:
        assert call(**kw) == BAD, kw
    assert call(hq=34) == UNS and call(pool=_pool(head_dim=256)) == UNS
    assert call(mb=1 << 27) == UNS and call(batch=70000) == UNS and call(total=1 << 31) == UNS
    assert call(pool=_pool(k_cache=0)) == BAD


def test_tree_refusals(lib):
    def call(pool=_pool(), **kw):
        a = dict(layer=0, q=16, hq=4, scale=0.1, bt=16, mb=4, lens=16, offs=None, cu=16, batch=2,
                 total=6, most=4, mask=16, words=1, qpos=16, window=8, sink=1, out=16, ws=16,
                 bytes=1 << 40, stream=None)
        a.update(kw)
        return lib.pkv_decode_attention_tree(pool, *a.values())

    for kw in (dict(batch=0), dict(total=0), dict(most=0)):
        assert call(**kw) == S["PKV_OK"]
    for kw in COMMON + CU + [dict(words=0), dict(words=-1), dict(most=65), dict(most=129, words=2),
                             dict(mask=None), dict(mask=None, words=0), dict(mask=12),
                             dict(mask=None, words=1, qpos=None), dict(qpos=2)]:
        assert call(**kw) == BAD, kw
    assert call(ws=0) == WS and call(ws=8) == WS
    assert call(hq=34) == UNS and call(pool=_pool(head_dim=256)) == UNS
    assert call(mb=1 << 27) == UNS and call(batch=70000) == UNS
    assert lib.pkv_decode_tree_workspace_size(_pool(), 2, 3, 4) == 0
    assert lib.pkv_decode_tree_workspace_size(_pool(head_dim=96), 2, 4, 4) == 0
    assert lib.pkv_decode_tree_workspace_size(_pool(), -1, 4, 4) == 0


def test_accept_refusals(lib):
    def call(pool=_pool(), **kw):
        a = dict(layer=-1, bt=16, mb=4, lens=16, offs=None, cu=16, batch=2, path=16, most=4, cnt=16,
                 stream=None)
        a.update(kw)
        return lib.pkv_accept_tokens(pool, *a.values())

    assert call(batch=0) == S["PKV_OK"] and call(most=0) == S["PKV_OK"]
    for kw in (dict(layer=2), dict(layer=-2), dict(batch=-1), dict(most=-1), dict(bt=0), dict(mb=0),
               dict(lens=0), dict(cu=0), dict(path=0), dict(cnt=0), dict(bt=2), dict(lens=2),
               dict(offs=2), dict(cu=4), dict(path=2), dict(cnt=2)):
        assert call(**kw) == BAD, kw
    assert call(mb=1 << 27) == UNS
    assert call(pool=_pool(k_cache=0)) == BAD


# ---- refusals of the binding ------------------------------------------------------

def test_binding_refusals():
    import torch

    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    pool = pkv.Pool(torch.zeros(4, 1, 16, 2, 64), torch.zeros(4, 1, 16, 2, 64))
    q, out, ws = torch.zeros(3, 4, 64), torch.zeros(3, 4, 64), torch.zeros(64)
    cu, mask = torch.zeros(3, dtype=torch.int64), torch.zeros(3, 1, dtype=torch.int64)
    good = dict(bt=i(2, 4), lens=i(2), offs=None, cu=cu, q=q, out=out, mask=mask, qpos=i(3), ws=ws,
                path=i(2, 5), count=i(2))
    bad = [dict(bt=i(8)), dict(bt=i(2, 4).long()), dict(lens=i(3)), dict(lens=i(2, 1)),
           dict(offs=i(3)), dict(offs=i(2).float())]
    cus = [dict(cu=cu[:2]), dict(cu=cu.int()), dict(cu=torch.zeros(6, dtype=torch.int64)[::2])]
    rows = [dict(q=q[0]), dict(q=q.half()), dict(out=out[:2]), dict(out=torch.zeros(3, 8, 64)[:, ::2]),
            dict(out=torch.zeros(3, 64, 4).transpose(1, 2)), dict(out=torch.zeros(6, 4, 64)[::2])]
    trees = [dict(mask=mask[:2]), dict(mask=mask.int()), dict(mask=mask[0]),
             dict(mask=torch.zeros(3, 0, dtype=torch.int64)), dict(qpos=i(2)), dict(mask=None),
             dict(ws=torch.zeros(64)[::2])]
    paths = [dict(path=i(5)), dict(path=i(3, 5)), dict(count=i(3)), dict(count=i(2).long())]

    def window(a):
        pkv.decode_attention_window(pool, 0, a["q"], 0.1, a["bt"], a["lens"], a["offs"], 4, a["out"])

    def prefill(a):
        pkv.prefill_attention_window(pool, 0, a["q"], 0.1, a["bt"], a["lens"], a["offs"], a["cu"], 3, 4,
                                     a["out"])

    def tree(a):
        pkv.decode_attention_tree(pool, 0, a["q"], 0.1, a["bt"], a["lens"], a["offs"], a["cu"], 3,
                                  a["mask"], a["out"], a["ws"], q_pos=a["qpos"])

    def accept(a):
        pkv.accept_tokens(pool, -1, a["bt"], a["lens"], a["offs"], a["cu"], a["path"], a["count"])

    two = dict(q=q[:2].contiguous(), out=out[:2].contiguous())
    for call, cases, base in ((window, bad + [dict(q=q, out=out)], two),
                              (prefill, bad + cus + rows, {}),
                              (tree, bad + cus + rows + trees, {}), (accept, bad + cus + paths, {})):
        for kw in cases + [{}]:  # (host tensors: refused too)
            with pytest.raises(ValueError):
                call({**good, **base, **kw})
