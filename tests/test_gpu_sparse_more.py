"""Sparse decode where one launch's work is more than its warps, calls of several
host threads, first calls inside a capture, dense attention at a bound that one row
would pass, the longest tables and positions, validate mode and empty batches."""

import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

from oracle import sparse as SP
import paged_kv_cache_blk_gb300 as pkv
from workloads import rand_rows

from gpu_util import dev_batch, gpu_decode, need_gpu, widen_out
from test_gpu_sparse import _case, _check_bounds, _layer_values, _queries, _random_bounds, _t

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    d = need_gpu()
    pkv.set_validate(False)
    pkv.device_error(clear=True)
    return d


@pytest.mark.parametrize("dtype,H,D,bs", [
    ("bf16", 7, 64, 16), ("bf16", 8, 128, 8), ("bf16", 1, 64, 4), ("f32", 3, 128, 8), ("f32", 5, 64, 16),
    ("i8", 7, 64, 8), ("i8", 3, 128, 16),
])
def test_bounds_of_more_blocks_than_warps(dev, dtype, H, D, bs):
    """One long sequence in a batch of many: its (block, head) pairs are several
    for each warp that the launch gives a sequence (46 CTAs of 4 on 152 SMs)."""
    blocks = max(100, 700 // H)
    lens = [blocks * bs - 3] + [3] * 39
    w, spec, pool = _case(dev, dtype, H, D, bs, lens, 171)
    bt, ln, offs, _ = dev_batch(w.batch, dev)
    kvals = _layer_values(pool.k_cache, spec, w.layer)
    bounds = pkv.BlockBounds.for_pool(pool)
    for first in (None, np.array([bs + 1] + [0] * 39)):
        bounds.codes.fill_(7)
        bounds.scales.fill_(-3.0)
        before = bounds.codes.cpu().numpy(), bounds.scales.cpu().numpy()
        pkv.update_block_bounds(pool, w.layer, bounds, bt, ln, offs,
                                None if first is None else _t(first, dev))
        assert _check_bounds(bounds, before, w, spec, kvals, first) * H > 46 * 4
    # an invalid block in the middle: it alone is skipped
    bounds.codes.fill_(7)
    bounds.scales.fill_(-3.0)
    before = bounds.codes.cpu().numpy(), bounds.scales.cpu().numpy()
    bad, at = bt.clone(), blocks // 2
    bad[0, at] = -1
    pkv.update_block_bounds(pool, w.layer, bounds, bad, ln, offs)
    assert pkv.device_error() == "PKV_ERR_INDEX"
    skipped = int(w.batch.block_tables[0, at])
    assert bool((bounds.codes[skipped] == 7).all())
    pkv.update_block_bounds(pool, w.layer, bounds, bt, ln, offs, _t([at * bs] + [5] * 39, dev))
    _check_bounds(bounds, before, w, spec, kvals)
    assert pkv.device_error() == "PKV_OK"


def test_calls_of_several_threads(dev):
    """Every thread's calls, on its own stream and with shapes of its own, give what
    they give alone."""
    jobs = []
    for i, (dtype, H, G, D, lens, K) in enumerate([
            ("bf16", 2, 4, 128, [900, 70], 9), ("f32", 1, 3, 64, [2000], 40),
            ("i8", 4, 2, 128, [300] * 20, 12), ("bf16", 1, 16, 64, [3000], 100),
            ("f32", 2, 9, 128, [500, 1], 6), ("i8", 1, 12, 64, [800], 50)]):
        w, spec, pool = _case(dev, dtype, H, D, 16, lens, 181 + i)
        rng = np.random.default_rng(190 + i)
        seq, pos = _queries(rng, lens, 2)
        bt, ln, offs, _ = dev_batch(w.batch, dev)
        q = rand_rows((len(seq), H * G, D), "f32" if dtype == "f32" else "bf16", 200 + i, dev)
        jobs.append((pool, w.layer, bt, ln, offs, _t(seq, dev), _t(pos, dev), q, H, K))
    torch.cuda.synchronize()

    def work(job):
        pool, layer, bt, ln, offs, seq, pos, q, H, K = job
        b = pkv.BlockBounds.for_pool(pool)
        sel = torch.full((len(seq), H, K), -7, dtype=torch.int32, device=dev)
        cnt = torch.full((len(seq), H), -7, dtype=torch.int32, device=dev)
        out = torch.full_like(q, 7.0)
        pkv.update_block_bounds(pool, layer, b, bt, ln, offs)
        pkv.select_blocks(pool, layer, b, q, bt, offs, seq, pos, sel, cnt, sink=1, recent=1)
        pkv.decode_attention_sparse(pool, layer, q, 0.1, bt, offs, seq, pos, sel, out)
        return sel, cnt, out

    alone = [[x.clone() for x in work(j)] for j in jobs]
    torch.cuda.synchronize()
    bad = []

    def run(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(8):
                    got = work(jobs[i])
                    torch.cuda.current_stream().synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, alone[i])):
                        bad.append((i, "differs"))
        except Exception as e:  # noqa: BLE001 - a thread's failure has to reach the test
            bad.append((i, repr(e)))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad and pkv.device_error() == "PKV_OK"


_CAPTURE = """
import torch
import paged_kv_cache_blk_gb300 as pkv
dev = torch.device("cuda", 0)
torch.manual_seed(1)
N, bs, H, D, G = 64, 16, 2, 128, 4
k = torch.randn(N, 1, bs, H, D, device=dev).bfloat16()
v = torch.randn_like(k)
pool = pkv.Pool(k, v)
b = pkv.BlockBounds.for_pool(pool)
i = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
bt = torch.randperm(N, device=dev).int()[:40].reshape(1, 40).contiguous()
ln, seq, pos = i([600]), i([0]), i([599])
q = torch.randn(1, H * G, D, device=dev).bfloat16()
kn, vn = (torch.randn(1, H, D, device=dev).bfloat16() for _ in range(2))
qr, out = torch.zeros_like(q), torch.zeros_like(q)
sel = torch.zeros(1, H, 8, dtype=torch.int32, device=dev)
cnt = torch.zeros(1, H, dtype=torch.int32, device=dev)
rope = pkv.Rope(D)

def step():
    pkv.rope_append(pool, 0, rope, bt, None, seq, pos, q, kn, vn, qr)
    pkv.update_block_bounds(pool, 0, b, bt, ln, None)
    pkv.select_blocks(pool, 0, b, qr, bt, None, seq, pos, sel, cnt, sink=1)
    pkv.decode_attention_sparse(pool, 0, qr, 0.1, bt, None, seq, pos, sel, out)

torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    step()
g.replay()
torch.cuda.synchronize()
a = [x.clone() for x in (qr, k, sel, cnt, out)]
assert a[0].any() and a[4].any() and int(a[3][0, 0]) == 8
step()
torch.cuda.synchronize()
assert all(torch.equal(x, y) for x, y in zip(a, (qr, k, sel, cnt, out)))
assert pkv.device_error() == "PKV_OK"
"""


def test_first_calls_of_a_process_inside_a_capture(dev):
    r = subprocess.run([sys.executable, "-c", _CAPTURE], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("dtype,D", [("f32", 64), ("f32", 128)])
def test_every_entry_is_dense_attention(dev, dtype, D):
    """Both calls in fp32 differ by their roundings alone: with A the weighted mean of
    |V| and S the largest sum of |q| |k| over n keys, 2 (2^-23 scale (D + 8) S + 2^-21) A +
    n 2^-23 A + 2^-24 |out| each.  One row of 900 left out changes an element by about
    1e-3, thousands of times that."""
    H, G, bs, lens = 4, 4, 16, [900, 37, 512, 1]
    w, spec, pool = _case(dev, dtype, H, D, bs, lens, 211)
    bt, ln, offs, _ = dev_batch(w.batch, dev)
    q = rand_rows((4, H * G, D), dtype, 212, dev)
    scale = D ** -0.5
    dense = gpu_decode(pool, w.layer, q, scale, w.batch, dev)
    sel = torch.arange(bt.shape[1], dtype=torch.int32, device=dev).expand(4, H, -1).contiguous()
    out = torch.empty_like(q)
    pkv.decode_attention_sparse(pool, w.layer, q, scale, bt, offs,
                                torch.arange(4, dtype=torch.int32, device=dev), ln - 1, sel, out)
    k, v = (_layer_values(c, spec, w.layer).astype(np.float64) for c in (pool.k_cache, pool.v_cache))
    x, got, want = widen_out(q).astype(np.float64), widen_out(out), widen_out(dense)
    for b, n in enumerate(lens):
        p = int(w.batch.offsets[b]) + np.arange(n)
        at = (w.batch.block_tables[b][p // bs], p % bs)
        for h in range(H * G):
            K, V = k[at][:, h // G], v[at][:, h // G]
            s = K @ x[b, h] * scale
            wt = np.exp(s - s.max())
            mean = wt / wt.sum() @ np.abs(V)
            top = (np.abs(K) @ np.abs(x[b, h])).max()
            tol = 2 * ((2 * (2.0 ** -23 * scale * (D + 8) * top + 2.0 ** -21) + n * 2.0 ** -23) * mean
                       + 2.0 ** -24 * np.abs(want[b, h]))
            assert np.all(np.abs(got[b, h].astype(np.float64) - want[b, h]) <= tol), (b, h)


@pytest.mark.parametrize("dtype,H,G,D", [("bf16", 2, 4, 128), ("f32", 1, 6, 64), ("i8", 2, 12, 64),
                                         ("i8", 3, 4, 128)])
def test_a_list_of_padding_and_of_one_query_many_times(dev, dtype, H, G, D):
    """The same query listed again gives the same bits; padding alone writes nothing."""
    w, spec, pool = _case(dev, dtype, H, D, 16, [700, 5], 221)
    rng = np.random.default_rng(222)
    bt, ln, offs, _ = dev_batch(w.batch, dev)
    T = 40
    q = rand_rows((1, H * G, D), "f32" if dtype == "f32" else "bf16", 223, dev).repeat(T, 1, 1)
    bounds = _random_bounds(pool, rng, dev, False)
    seq, pos = np.zeros(T, np.int32), np.full(T, 650, np.int32)
    sel = torch.empty((T, H, 20), dtype=torch.int32, device=dev)
    cnt = torch.empty((T, H), dtype=torch.int32, device=dev)
    out = torch.empty_like(q)
    pkv.select_blocks(pool, w.layer, bounds, q, bt, offs, _t(seq, dev), _t(pos, dev), sel, cnt)
    pkv.decode_attention_sparse(pool, w.layer, q, 0.1, bt, offs, _t(seq, dev), _t(pos, dev), sel, out)
    assert torch.equal(sel, sel[:1].expand_as(sel)) and torch.equal(out, out[:1].expand_as(out))
    before = out.clone()
    pad = _t(np.full(T, -3), dev)
    pkv.select_blocks(pool, w.layer, bounds, q, bt, offs, pad, _t(pos, dev), sel, cnt)
    pkv.decode_attention_sparse(pool, w.layer, q, 0.1, bt, offs, pad, _t(pos, dev), sel, out)
    assert torch.equal(out, before) and bool((sel == -1).all()) and not cnt.any()
    assert pkv.device_error() == "PKV_OK"


@pytest.mark.parametrize("n,K", [(327680, 500), (327679, 3), (200001, 200000)])
def test_the_longest_tables(dev, n, K):
    """As many entries as a selection takes, over blocks that repeat (equal scores)."""
    N, D, G = 911, 64, 3
    rng = np.random.default_rng(231)
    pool = pkv.Pool(*(torch.zeros((N, 1, 1, 1, D), dtype=torch.bfloat16, device=dev) for _ in range(2)))
    bounds = _random_bounds(pool, rng, dev, False)
    table = rng.integers(0, N, (1, 327680)).astype(np.int32)
    q = rand_rows((1, G, D), "bf16", 232, dev)
    sel = torch.empty((1, 1, K), dtype=torch.int32, device=dev)
    cnt = torch.empty((1, 1), dtype=torch.int32, device=dev)
    one = lambda x: torch.tensor([x], dtype=torch.int32, device=dev)
    pkv.select_blocks(pool, 0, bounds, q, _t(table, dev), None, one(0), one(n - 1), sel, cnt, sink=1,
                      recent=2)
    codes = bounds.codes.cpu().numpy().astype(np.int64) - 128
    score = SP.block_scores(widen_out(q)[0], codes[:, 0, 0], bounds.scales.cpu().numpy()[:, 0, 0])
    want = SP.select(score[table[0, :n]], K, 1, 2)
    assert int(cnt[0, 0]) == K and np.array_equal(sel[0, 0].cpu().numpy(), want)
    assert pkv.device_error() == "PKV_OK"


@pytest.mark.parametrize("dtype", ["bf16", "f32", "i8"])
def test_positions_near_two_to_the_thirty(dev, dtype):
    """Table entries far out: the rotary append, the bounds of the last blocks and
    the attention over them find the rows that a short table of the same blocks names."""
    H, G, D, bs, MB = 2, 3, 64, 1024, 1 << 20
    w, spec, pool = _case(dev, dtype, H, D, bs, [2500], 241, offsets=False)
    ids = w.batch.block_tables[0, :3]
    far = np.full((1, MB), -1, np.int32)
    far[0, -3:] = ids
    shift = (MB - 3) * bs
    near = np.ascontiguousarray(ids[None])
    one = lambda x: torch.tensor([x], dtype=torch.int32, device=dev)
    io = "f32" if dtype == "f32" else "bf16"
    q, k, v = (rand_rows((1, h, D), io, 242 + h, dev) for h in (H * G, H, H))
    k0, v0 = pool.k_cache.clone(), pool.v_cache.clone()
    got = []
    for table, base in ((near, 0), (far, shift)):
        pool.k_cache.copy_(k0)
        pool.v_cache.copy_(v0)
        bt, last = _t(table, dev), base + 2999
        b = pkv.BlockBounds.for_pool(pool)
        b.codes.fill_(0)
        b.scales.fill_(0)
        qr, out = torch.zeros_like(q), torch.zeros_like(q)
        pkv.rope_append(pool, w.layer, pkv.Rope(D), bt, None, one(0), one(last), q, k, v, qr,
                        rope_pos=one(7))
        pkv.update_block_bounds(pool, w.layer, b, bt, one(last + 1), None, one(base + 1500))
        e = base // bs
        sel = torch.tensor([[[e + 2, -1, e + 1], [e, e + 2, e + 1]]], dtype=torch.int32, device=dev)
        # (the far table's first rows are no blocks: positions from `shift` on are listed)
        pkv.decode_attention_sparse(pool, w.layer, q, 0.1, bt, None, one(0), one(last), sel, out)
        got.append((qr, pool.k_cache.clone(), pool.v_cache.clone(), b.codes, b.scales, out))
        assert pkv.device_error() == "PKV_OK"
    assert all(torch.equal(x, y) for x, y in zip(*got))
    assert not torch.equal(got[0][1], k0) and got[0][5].any()


@pytest.mark.parametrize("dtype", ["bf16", "i8"])
def test_validate_mode(dev, dtype):
    """Every call with valid inputs passes its validation and gives what it gives
    without; a bad token or table is refused with nothing written."""
    H, G, D, bs = 2, 4, 64, 16
    w, spec, pool = _case(dev, dtype, H, D, bs, [300, 41], 251)
    bt, ln, offs, _ = dev_batch(w.batch, dev)
    q, k, v = (rand_rows((3, h, D), "bf16", 252 + h, dev) for h in (H * G, H, H))
    seq, pos = _t([0, -1, 1], dev), _t([299, 0, 40], dev)

    def calls(seq, bt):
        b = pkv.BlockBounds.for_pool(pool)
        b.codes.fill_(0)
        b.scales.fill_(0)
        qr, out = (torch.full_like(q, 7.0) for _ in range(2))
        sel = torch.full((3, H, 5), 77, dtype=torch.int32, device=dev)
        cnt = torch.full((3, H), 77, dtype=torch.int32, device=dev)
        return (qr, b.codes, sel, cnt, out), (
            lambda: pkv.rope_append(pool, w.layer, pkv.Rope(D), bt, offs, seq, pos, q, k, v, qr),
            lambda: pkv.update_block_bounds(pool, w.layer, b, bt, ln, offs),
            lambda: pkv.select_blocks(pool, w.layer, b, q, bt, offs, seq, pos, sel, cnt),
            lambda: pkv.decode_attention_sparse(pool, w.layer, q, 0.1, bt, offs, seq, pos, sel, out))

    plain, run = calls(seq, bt)
    for f in run:
        f()
    pkv.set_validate(True)
    try:
        checked, run = calls(seq, bt)
        for f in run:
            f()
        assert all(torch.equal(x, y) for x, y in zip(plain, checked))
        bad_table = bt.clone()
        bad_table[0] = spec.num_blocks
        for s, t in ((_t([2, -1, 1], dev), bt), (seq, bad_table)):
            before = pool.k_cache.clone()
            outs, run = calls(s, t)
            for i, f in enumerate(run):
                if i == 1 and t is bt:
                    continue  # (the bounds take no token list)
                with pytest.raises(pkv.PkvError) as e:
                    f()
                assert e.value.name == "PKV_ERR_INDEX"
            assert torch.equal(pool.k_cache, before) and bool((outs[4] == 7).all())
            assert bool((outs[2] == 77).all()) and not outs[1].any()
    finally:
        pkv.set_validate(False)
    assert pkv.device_error() == "PKV_OK"


def test_no_sequences_at_all(dev):
    """A table without rows: padding is passed over, any other token is an error."""
    w, spec, pool = _case(dev, "bf16", 2, 64, 16, [40], 261)
    none = torch.empty((0, 4), dtype=torch.int32, device=dev)
    empty = torch.empty((0,), dtype=torch.int32, device=dev)
    q, k = rand_rows((2, 4, 64), "bf16", 262, dev), rand_rows((2, 2, 64), "bf16", 263, dev)
    bounds = pkv.BlockBounds.for_pool(pool)
    before = pool.k_cache.clone()
    for first, want in ((-1, "PKV_OK"), (0, "PKV_ERR_INDEX")):
        seq, pos = _t([first, -1], dev), _t([0, 0], dev)
        sel = torch.full((2, 2, 3), 77, dtype=torch.int32, device=dev)
        cnt = torch.full((2, 2), 77, dtype=torch.int32, device=dev)
        out = torch.full_like(q, 7.0)
        pkv.rope_append(pool, 0, pkv.Rope(64), none, empty, seq, pos, q, k, k, out)
        assert bool((out == 7).all()) and pkv.device_error() == want
        pkv.update_block_bounds(pool, 0, bounds, none, empty, empty)
        pkv.select_blocks(pool, 0, bounds, q, none, empty, seq, pos, sel, cnt)
        assert not cnt.any() and bool((sel == -1).all()) and pkv.device_error() == want
        pkv.decode_attention_sparse(pool, 0, q, 0.1, none, empty, seq, pos, sel, out)
        assert bool((out[1] == 7).all()) and bool((out[0] == (7 if first < 0 else 0)).all())
        assert pkv.device_error() == want
    assert torch.equal(pool.k_cache, before)
