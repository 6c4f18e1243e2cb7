"""Table entries of windowed calls and trees: any id outside the pool is an error where a query sees a
key of its block, and no entry matters whose block holds no seen key."""

import numpy as np
import pytest
import torch

import paged_kv_cache_blk_gb300 as pkv
from oracle import masked as MK
from paged_kv_cache_blk_gb300 import PkvError

from gpu_util import need_gpu
from test_gpu_masked import Case, _prefill, _tree, _tree_args, _weight_err, _window

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    d = need_gpu()
    pkv.set_validate(False)
    pkv.device_error(clear=True)
    return d


@pytest.fixture
def window_path():
    yield pkv.set_debug_window_path
    pkv.set_debug_window_path(0)


def _both(call, error):
    """Without validate mode the error word says ``error``, with it the call does."""
    call()
    assert pkv.device_error() == error
    pkv.set_validate(True)
    try:
        if error == "PKV_OK":
            call()
        else:
            with pytest.raises(PkvError) as e:
                call()
            assert e.value.name == error
    finally:
        pkv.set_validate(False)
    assert pkv.device_error() == "PKV_OK"


@pytest.mark.parametrize("bad", [-(1 << 31), -(1 << 31) + 1, -1, (1 << 31) - 1, "blocks"])
@pytest.mark.parametrize("what,dtype,D", [
    ("window", "bf16", 128), ("window", "f32", 64), ("window", "i8", 64), (1, "bf16", 128), (1, "f32", 64),
    (1, "i8", 128), (2, "bf16", 128), (2, "bf16", 64), ("tree", "bf16", 128), ("tree", "bf16", 64),
    ("tree", "f32", 128), ("tree", "i8", 64), ("few", "bf16", 128), ("few", "i8", 128)])
def test_ids_outside_the_pool(dev, window_path, what, dtype, D, bad):
    """Every id outside the pool, the lowest of the type among them, is reported and reads as zeros (the
    single-token call, as pkv_decode_attention, leaves its keys out)."""
    n = 1 if what == "window" else 3 if what == "few" else 30
    c = Case(dev, dtype, 2, 4, D, 16, [100, 60], [n, n], seed=71, offsets=False)
    c.table[0, 5] = c.spec.num_blocks if bad == "blocks" else bad
    if what in (1, 2):
        window_path(what)
    mask, pos = _tree_args(c, [np.tril(np.ones((n, n)))] * 2, [np.arange(n)] * 2, 1)
    call = {"window": lambda: _window(c, 50, 3), "tree": lambda: _tree(c, mask, pos),
            "few": lambda: _tree(c, None, None)}.get(what, lambda: _prefill(c, 50, 3))
    # keys 80 to 95 read as zeros
    kv = c.values(c.k), c.values(c.v)
    blk = int(c.home[0, 5])
    for x in kv:
        x[blk] = 0.0
    got = call()
    assert pkv.device_error() == "PKV_ERR_INDEX"

    def seen_of(b, i):
        s = MK.window_seen(int(c.lens[b] - n) + i, 50 if what in ("window", 1, 2) else 0, 3)
        if what == "window" and b == 0:
            s[80:96] = False
        return s

    c.check(got, *kv, seen_of, _weight_err(dtype, n * 4 > 16), fma=what == "window")
    _both(call, "PKV_ERR_INDEX")


@pytest.mark.parametrize("dtype,G,D,bs,n", [
    ("bf16", 4, 128, 16, 40), ("bf16", 4, 128, 16, 6), ("bf16", 2, 128, 16, 100), ("bf16", 4, 64, 16, 20),
    ("bf16", 4, 64, 4, 20), ("f32", 3, 64, 8, 30), ("i8", 4, 128, 16, 24), ("i8", 2, 64, 16, 4)])
def test_entries_that_no_query_of_a_tree_sees(dev, dtype, G, D, bs, n):
    """Positions that all lie above the context's end leave its oldest window tokens behind, and bits
    that no row sets hide drafted tokens: entries of blocks with nothing else may hold anything."""
    window, sink, ctx = 50, 3, 150
    c = Case(dev, dtype, 2, G, D, bs, [ctx + n, 70 + n], [n, n], seed=72)
    kv = c.values(c.k), c.values(c.v)
    sees = np.tril(np.ones((n, n), bool))
    hidden = slice(n // 3, n // 3 + max(1, n // 2))
    sees[:, hidden] = False
    depth = np.arange(n) + 45  # (the windows begin in the context for the first five tokens)
    mask, pos = _tree_args(c, [sees, sees], [depth, depth], -(-n // 64))

    def seen_of(b, i):
        at = int(c.lens[b] - n)
        return MK.tree_seen(at, sees, i, at + int(depth[i]), window, sink)

    some = []
    for b in range(2):
        s = np.zeros(int(c.lens[b]), bool)
        for i in range(n):
            s |= seen_of(b, i)
        some.append(s)
    c.poison(some)
    call = lambda: _tree(c, mask, pos, window, sink)
    got = call()
    assert pkv.device_error() == "PKV_OK"
    c.check(got, *kv, seen_of, _weight_err(dtype, n * G > 16))
    _both(call, "PKV_OK")
    # the block of the first token that only some rows see
    b_seen = int(c.offs[0] + ctx + n - 1) // bs
    c.table[0, b_seen] = -1
    _both(call, "PKV_ERR_INDEX")
    c.table[0, b_seen] = c.home[0, b_seen]
    c.table[1, 0] = 1 << 30
    _both(call, "PKV_ERR_INDEX")
