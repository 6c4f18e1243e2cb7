"""Values that some queries see and others do not, on each kernel that multiplies them: what a
query does not see never reaches its result, and computing spoiled results again holds up no
launch.  Tolerances: those of test_gpu_masked.py, whose oracle the repaired rows are held to."""

import numpy as np
import pytest
import torch

import paged_kv_cache_blk_gb300 as pkv
from oracle import masked as MK
from paged_kv_cache_blk_gb300 import PkvError

from gpu_util import need_gpu
from test_gpu_masked import Case, _prefill, _random_tree, _t, _tree, _tree_args, _weight_err

pytestmark = pytest.mark.gpu

MMA, TCGEN05 = 1, 2  # pkv.set_debug_window_path


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


def test_the_path_hook(dev, window_path):
    """A pool that the asked-for kernel cannot take is refused, so a call that returns took it."""
    for bad in (-1, 3):
        with pytest.raises(PkvError) as e:
            window_path(bad)
        assert e.value.name == "PKV_ERR_INVALID_ARG"
    c = Case(dev, "f32", 1, 2, 64, 16, [40], [40])
    want = _prefill(c, 10, 1)
    window_path(MMA)
    assert torch.equal(_prefill(c, 10, 1), want)
    window_path(TCGEN05)
    with pytest.raises(PkvError) as e:
        _prefill(c, 10, 1)
    assert e.value.name == "PKV_ERR_UNSUPPORTED"


def _spoil(c, b, j, bad):
    """V of new token j of sequence b, in both kv heads, to ``bad``."""
    place = int(c.offs[b] + c.lens[b] - c.new[b]) + j
    blk, row = int(c.home[b, place // c.bs]), place % c.bs
    if c.dtype == "i8":
        at = c.H * c.D
        c.v[blk, c.layer, row, at:at + 4 * c.H].view(torch.float32).fill_(bad)
    else:
        c.v[blk, c.layer, row] = bad


def _check_spoiled(c, run, seen_of, j_of, bad, one_part):
    """``run()`` clean, then with V of token j_of[b] of each listed sequence bad: the rows that see it
    are not finite, all others are the oracle's."""
    kv = c.values(c.k), c.values(c.v)
    clean = run()
    for b, j in j_of.items():
        _spoil(c, b, j, bad)
    got = run().clone()
    for b, j in j_of.items():
        for i in range(int(c.new[b])):
            s = seen_of(b, i)
            at = int(c.lens[b] - c.new[b]) + j
            if at < len(s) and s[at]:
                t = int(c.cu[b]) + i
                assert not bool(got[t].isfinite().any()) or c.dtype == "i8", (b, i)
                got[t] = clean[t]
    c.check(got, *kv, seen_of, _weight_err(c.dtype, one_part))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("path,dtype,G,D,lens,new", [
    (TCGEN05, "bf16", 4, 128, [300], [40]), (TCGEN05, "bf16", 4, 128, [900, 70], [300, 3]),
    (TCGEN05, "bf16", 3, 64, [700, 41], [150, 41]), (TCGEN05, "bf16", 1, 128, [600], [520]),
    (TCGEN05, "bf16", 16, 64, [260, 33], [70, 33]),
    (TCGEN05, "bf16", 2, 128, [70 + 5 * i for i in range(60)], [30 + 3 * i for i in range(60)]),
    (MMA, "bf16", 4, 128, [900, 70], [300, 3]), (MMA, "f32", 3, 64, [200, 40], [60, 3]),
    (MMA, "i8", 4, 128, [300, 70], [40, 3]), (MMA, "bf16", 2, 64, [3000], [5])])
def test_windowed_prompts(dev, window_path, path, dtype, G, D, lens, new, bad):
    """Under a window of 9, one token of the first and of the last sequence (60 sequences: of the
    last alone, in items beyond the first of a CTA pair) is seen by nine queries at most."""
    window_path(path)
    c = Case(dev, dtype, 2, G, D, 16, lens, new, seed=61)
    j_of = {len(lens) - 1: int(new[-1]) // 2}
    if len(lens) < 60:
        j_of[0] = new[0] // 3
    _check_spoiled(c, lambda: _prefill(c, 9, 2),
                   lambda b, i: MK.window_seen(int(c.lens[b] - c.new[b]) + i, 9, 2), j_of, bad,
                   max(new) * G > 16)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype,G,D,n,batch", [
    ("bf16", 4, 128, 20, 2), ("bf16", 4, 128, 20, 100), ("bf16", 4, 128, 60, 2), ("bf16", 4, 128, 60, 100),
    ("bf16", 3, 64, 30, 100), ("bf16", 3, 64, 80, 100), ("bf16", 4, 128, 3, 200), ("f32", 2, 64, 5, 100),
    ("f32", 1, 128, 20, 3), ("i8", 4, 64, 6, 200)])
def test_trees(dev, dtype, G, D, n, batch, bad):
    """Few sequences: states of split units, repaired by their merge; many: units that a CTA finishes."""
    c = Case(dev, dtype, 2, G, D, 16, [150 + n + 3 * (i % 40) for i in range(batch)], [n] * batch, seed=62)
    made = [_random_tree(c.rng, n) for _ in range(batch)]
    mask, pos = _tree_args(c, [t for t, _ in made], [d for _, d in made], -(-n // 64))

    def seen_of(b, i):
        ctx = int(c.lens[b] - n)
        return MK.tree_seen(ctx, made[b][0], i, ctx + int(made[b][1][i]), 0, 0)

    _check_spoiled(c, lambda: _tree(c, mask, pos), seen_of, {0: n // 2, batch - 1: 0}, bad, n * G > 16)


@pytest.mark.parametrize("what,G,D,n", [("prefill", 4, 128, 64), ("prefill", 2, 64, 200), ("narrow", 4, 64, 20),
                                        ("narrow", 4, 128, 20), ("tree", 4, 128, 50)])
def test_no_wait_runs_out_on_it(dev, window_path, what, G, D, n):
    """An infinity in the V row of a long context's last token, which other tokens do not see, with the
    bound of a wait at 10 ms: the launch ends without a timeout, and sequences that hold nothing wrong
    have their results to the bit."""
    window_path(TCGEN05)
    H, bs, ctx, batch = 4, 16, 20000, 48
    N = (ctx + n + bs - 1) // bs
    gen = torch.Generator(device=dev)
    gen.manual_seed(7)
    k, v = (torch.randn((N + 1, 1, bs, H, D), generator=gen, device=dev).bfloat16() for _ in range(2))
    k[N], v[N] = k[N - 1], v[N - 1]
    pool = pkv.Pool(k, v)
    # every sequence reads the same blocks, but for the last, of which odd ones have a copy
    table = torch.arange(N, device=dev, dtype=torch.int32).repeat(batch, 1)
    table[1::2, N - 1] = N
    lens = torch.full((batch,), ctx + n, device=dev, dtype=torch.int32)
    q = torch.randn((batch * n, H * G, D), generator=gen, device=dev).bfloat16()
    cu = torch.arange(batch + 1, device=dev, dtype=torch.int64) * n
    out = torch.empty_like(q)
    ws = torch.empty(pkv.decode_tree_workspace_size(pool, batch, H * G, n), dtype=torch.uint8, device=dev)

    def run():
        if what == "prefill":
            pkv.prefill_attention_window(pool, 0, q, D ** -0.5, table, lens, None, cu, n, 1 << 20, out)
        else:
            pkv.decode_attention_tree(pool, 0, q, D ** -0.5, table, lens, None, cu, n, None, out, ws)
        return out.clone()

    clean = run()
    v[N - 1, 0, (ctx + n - 1) % bs] = float("inf")
    pkv.set_wait_limit_ns(10_000_000)
    try:
        got = run()
        assert pkv.device_error() == "PKV_OK"
    finally:
        pkv.set_wait_limit_ns(0)
    got, clean = (x.view(batch, n, H * G, D) for x in (got, clean))
    assert torch.equal(got[1::2], clean[1::2])
    assert not bool(got[::2, -1].isfinite().any())
    # computed another way: the weights of one result were rounded, 2^-9 of the mean |v| (below 0.85) if
    # all err to one side, and the output of each is, 2^-9 of an average (below 1/8) of 20000 values
    assert float((got[::2, :-1].float() - clean[::2, :-1].float()).abs().max()) <= 2.0 ** -8
