"""Scores of every kind under windows and in trees: far apart (so that a row's maximum rises within a
tile), scaled by a negative number or by zero, and NaN or infinite for some queries.

Tolerances: those of test_gpu_masked_paths.py.  On tcgen05 a weight whose tile of 128 keys holds a
later one more than 2^8 above the maximum so far is rounded twice: 2^-7."""

import numpy as np
import pytest
import torch

import paged_kv_cache_blk_gb300 as pkv
from oracle import masked as MK

from gpu_util import need_gpu
from test_gpu_masked import Case, _prefill, _random_tree, _tree, _tree_args, _window
from test_gpu_masked_paths import MMA, TCGEN05, _check_weights, _weight

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


def _tree_case(c):
    n = int(c.new.max())
    made = [_random_tree(c.rng, int(m)) for m in c.new]
    mask, pos = _tree_args(c, [t for t, _ in made], [d for _, d in made], -(-n // 64))

    def seen_of(b, i):
        ctx = int(c.lens[b] - c.new[b])
        return MK.tree_seen(ctx, made[b][0], i, ctx + int(made[b][1][i]), 0, 0)

    return (lambda: _tree(c, mask, pos)), seen_of


def _prompt_case(c, window=200, sink=3):
    return (lambda: _prefill(c, window, sink)), \
        lambda b, i: MK.window_seen(int(c.lens[b] - c.new[b]) + i, window, sink)


KINDS = [("tree", "bf16", 4, 128, 40), ("tree", "bf16", 4, 128, 10), ("tree", "bf16", 4, 128, 3),
         ("tree", "bf16", 3, 64, 50), ("tree", "bf16", 4, 64, 11), ("tree", "f32", 3, 64, 9), ("tree", "i8", 4, 128, 12),
         ("tree", "i8", 2, 64, 4), (TCGEN05, "bf16", 4, 128, 150), (TCGEN05, "bf16", 3, 64, 100),
         (MMA, "bf16", 4, 128, 100), (MMA, "f32", 2, 128, 20), (MMA, "i8", 4, 64, 40)]


def _case(dev, window_path, kind, dtype, G, D, n, seed=141):
    c = Case(dev, dtype, 2, G, D, 16, [400 + n, 60 + n // 2], [n, n // 2 + 1], seed=seed)
    if kind == "tree":
        return (c, *_tree_case(c))
    window_path(kind)
    return (c, *_prompt_case(c))


def _on_tcgen05(kind, dtype, G, D, n):
    return kind == TCGEN05 or (kind == "tree" and dtype == "bf16" and n * G > (16 if D == 128 else 32))


@pytest.mark.parametrize("scale", [1.0, -0.3, 0.0])
@pytest.mark.parametrize("kind,dtype,G,D,n", KINDS)
def test_scales(dev, window_path, kind, dtype, G, D, n, scale):
    """Scale 1: scores of a standard deviation of sqrt(D), 16 in log2 units for D 128."""
    c, run, seen_of = _case(dev, window_path, kind, dtype, G, D, n)
    c.scale = scale
    err = 2.0 ** -7 if _on_tcgen05(kind, dtype, G, D, n) else _weight(dtype, n * G > 16)
    c_abs = Case.__new__(Case)  # (the oracle's check takes the size of a score from a positive scale)
    c_abs.__dict__.update(c.__dict__)
    if scale < 0:
        c_abs.scale, c_abs.q = -scale, -c.q
    _check_weights(c_abs, run(), c.values(c.k), c.values(c.v), seen_of, err)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f32", 64), ("i8", 64)])
@pytest.mark.parametrize("scale", [1.0, -0.3, 0.0])
def test_window_decode_scales(dev, dtype, D, scale):
    c = Case(dev, dtype, 2, 4, D, 16, [400, 30], [1, 1], seed=142)
    c.scale = scale
    got = _window(c, 200, 3)
    if scale < 0:
        c.scale, c.q = -scale, -c.q
    c.check(got, c.values(c.k), c.values(c.v),
            lambda b, i: MK.window_seen(int(c.lens[b]) - 1, 200, 3), 2.0 ** -16 if dtype != "f32" else 3 * 2.0 ** -22,
            fma=True)


@pytest.mark.parametrize("rising", [True, False])
@pytest.mark.parametrize("kind,dtype,G,D,n", KINDS)
def test_a_maximum_that_moves(dev, window_path, kind, dtype, G, D, n, rising):
    """Scores that climb (or fall) along the keys by 0.2 in log2 units a key: the maximum is passed by
    2^8 again and again, within tiles and between them, and far keys end at weights of zero."""
    c, run, seen_of = _case(dev, window_path, kind, dtype, G, D, n)
    # q and k of one direction: dim 0 carries the key's place, the others little
    c.q.mul_(0.05)
    c.q[..., 0] = 8.0
    if dtype == "i8":
        at = c.k[..., :c.H * D].view(c.k.shape[:3] + (c.H, D))
        unit = c.k[..., c.H * D:c.H * D + 4 * c.H].view(torch.float32)
    for b in range(2):
        blk, row = c.rows(b)
        m = len(blk)
        place = (np.arange(m) if rising else m - 1 - np.arange(m)) * (0.2 * np.log(2.0) / (8.0 * c.scale))
        blk, row = (torch.from_numpy(np.asarray(x)).to(dev) for x in (blk, row))
        x = torch.from_numpy(place).to(dev)
        if dtype == "i8":
            unit[blk, c.layer, row] = (x / 127).clamp(min=1e-6).float()[:, None].expand(m, c.H)
            codes = torch.randint(126, 131, (m, c.H, D), device=dev, dtype=torch.uint8)
            codes[..., 0] = 255
            at[blk, c.layer, row] = codes
        else:
            c.k[blk, c.layer, row, :, 0] = x.to(c.k.dtype)[:, None].expand(m, c.H)
    err = 2.0 ** -7 if _on_tcgen05(kind, dtype, G, D, n) else _weight(dtype, n * G > 16)
    _check_weights(c, run(), c.values(c.k), c.values(c.v), seen_of, err)


@pytest.mark.parametrize("what", ["key", "query"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("kind,dtype,G,D,n", KINDS)
def test_bad_keys_and_queries_stay_with_their_rows(dev, window_path, kind, dtype, G, D, n, bad, what):
    """A key row of NaN or infinities reaches the queries that see it and no other; a query's reaches
    its own result alone.  All other results stay as they are."""
    c, run, seen_of = _case(dev, window_path, kind, dtype, G, D, n)
    clean = run()
    j = n // 2
    if what == "query":
        c.q[j] = bad
        hit = [i == j for i in range(n)]
    else:
        place = int(c.offs[0] + c.lens[0]) - n + j
        blk, row = int(c.home[0, place // 16]), place % 16
        if dtype == "i8":
            c.k[blk, c.layer, row, 2 * D:2 * D + 8].view(torch.float32).fill_(bad)
        else:
            c.k[blk, c.layer, row] = bad
        at = int(c.lens[0]) - n + j
        hit = [at < len(seen_of(0, i)) and bool(seen_of(0, i)[at]) for i in range(n)]
    got = run()
    hit = torch.tensor(hit + [False] * (len(got) - n), device=dev)
    assert bool(got[~hit].isfinite().all())
    # (mma.sync: where one row's maximum moves those of the unit are all agreed on anew, so to rounding: of
    # outputs below 1.5 twice 2^-8 and of weights twice 2^-8 of the mean |v|, below 0.85; fp32 2^-21 and sums)
    if _on_tcgen05(kind, dtype, G, D, n):
        assert torch.equal(got[~hit], clean[~hit])
    else:
        diff = float((got[~hit].float() - clean[~hit].float()).abs().max())
        assert diff <= (1e-5 if dtype == "f32" else 2.0 ** -5)
    if bad != bad:
        assert not bool(got[hit].isfinite().any())
    assert pkv.device_error() == "PKV_OK"
