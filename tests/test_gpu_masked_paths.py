"""Windowed prompts on each of their two kernels, weights held to the documented rounding, chains as
masks, and the uses that one call alone does not show: several host threads, first calls inside a
capture, far positions, pools past 2^32 bytes, the same bits every time.

Tolerances: those of test_gpu_masked.py, with what a weight's own rounding is documented to be.  One
bf16 part: the nearest of 8 significant bits, half a step of 2^-7 for a weight just above a power of
two, so torch.finfo(torch.bfloat16).eps / 2 = 2^-8 of it, and 2^-8 A.  int8: one fp16 part 2^-11 of each product of a
weight and a V scale, two 2^-22, or 2^-27 of the largest product of the row, times a code of up to
127, for each of n keys."""

import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import paged_kv_cache_blk_gb300 as pkv
import test_gpu_masked as base
from oracle import masked as MK
from workloads import rand_rows

from gpu_util import need_gpu, widen_out
from test_gpu_masked import Case, _prefill, _random_tree, _t, _tree, _tree_args, _window, _workspace

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


def _check_weights(c, got, kvals, vvals, seen_of, weight_err):
    """Case.check, with the documented error of a weight (int8: and of the row's largest product)."""
    D, G = c.D, c.G
    got, q = widen_out(got), widen_out(c.q)
    bf16 = c.dtype != "f32"
    for b in range(len(c.lens)):
        blk, row = c.rows(b)
        for g in range(c.H):
            k, v = kvals[blk, row, g], vvals[blk, row, g]
            for i in range(int(c.new[b])):
                t, seen = int(c.cu[b]) + i, seen_of(b, i)
                full = np.zeros(len(k), bool)
                full[:len(seen)] = seen
                rows = slice(g * G, (g + 1) * G)
                ref, mean, top = MK.attention(q[t, rows], k, v, full, c.scale)
                n = int(full.sum())
                d = (D + 8 if bf16 else 3 * D // 8 + 8) * 2.0 ** -23 * c.scale * top[:, None] + 2.0 ** -21
                tol = (2 * d + n * 2.0 ** -23 + weight_err) * mean
                if c.dtype == "i8" and n:
                    x = c.scale * (q[t, rows] @ k[full].T)
                    w = np.exp(x - x.max(1, keepdims=True))
                    most = (w / w.sum(1, keepdims=True) * (np.abs(v[full]).max(1) / 127)).max(1, keepdims=True)
                    tol += n * 127 * 2.0 ** -27 * most
                tol += np.abs(ref) * 1.01 * (2.0 ** -8 if bf16 else 2.0 ** -24)
                err = np.abs(got[t, rows] - ref)
                assert np.all(err <= tol + 1e-30), (b, i, g, float((err / (tol + 1e-30)).max()))
    assert pkv.device_error() == "PKV_OK"


def _weight(dtype, one_part):
    return {"f32": 3 * 2.0 ** -22, "bf16": 2.0 ** -8 if one_part else 2.0 ** -16,
            "i8": 2.0 ** -11 if one_part else 2.0 ** -22}[dtype]


def _seen_rows(c, seen_of):
    some = []
    for b in range(len(c.lens)):
        s = np.zeros(int(c.lens[b]), bool)
        for i in range(int(c.new[b])):
            x = seen_of(b, i)
            s[:len(x)] |= x
        some.append(s)
    return some


def _run_prefill(dev, dtype, H, G, D, bs, lens, new, window, sink, one_part, seed=4, most=None):
    c = Case(dev, dtype, H, G, D, bs, lens, new, seed, extra_blocks=seed % 3)
    kv = c.values(c.k), c.values(c.v)
    seen_of = lambda b, i: MK.window_seen(int(c.lens[b] - c.new[b]) + i, window, sink)
    c.poison(_seen_rows(c, seen_of))
    _check_weights(c, _prefill(c, window, sink, most), *kv, seen_of, _weight(dtype, one_part))


# ---- windowed prompts on the kernel that is asked for ------------------------------------

def _on_tcgen05(case):
    dtype, H, G, D, bs = case[:5]
    return dtype == "bf16" and 8 <= bs <= (64 if D == 64 else 128)


@pytest.mark.parametrize("dtype,H,G,D,bs,lens,new,window,sink", [x for x in base.PREFILLS if _on_tcgen05(x)] + [
    ("bf16", 1, 12, 128, 16, [300, 41], [200, 41], 90, 5), ("bf16", 2, 6, 64, 8, [260], [130], 1, 0),
    ("bf16", 1, 9, 64, 64, [500, 1], [129, 1], 1 << 30, 0), ("bf16", 1, 14, 128, 128, [300], [100], 40, 300),
    ("bf16", 3, 10, 64, 32, [129], [129], 31, 64), ("bf16", 1, 15, 128, 32, [90, 70], [1, 33], 33, 2),
    ("bf16", 2, 2, 64, 16, [2000, 700], [600, 1], 500, 100), ("bf16", 1, 1, 64, 64, [1300], [1300], 700, 4)])
def test_prompts_on_tcgen05(dev, window_path, dtype, H, G, D, bs, lens, new, window, sink):
    window_path(TCGEN05)
    _run_prefill(dev, dtype, H, G, D, bs, lens, new, window, sink, True)


@pytest.mark.parametrize("dtype,H,G,D,bs,lens,new,window,sink", base.PREFILLS)
def test_prompts_on_mma(dev, window_path, dtype, H, G, D, bs, lens, new, window, sink):
    window_path(MMA)
    _run_prefill(dev, dtype, H, G, D, bs, lens, new, window, sink, max(new) * G > 16)


@pytest.mark.parametrize("path", [MMA, TCGEN05])
@pytest.mark.parametrize("G,D,bs,seqs,tokens", [(4, 128, 16, 16, 300), (1, 64, 8, 16, 290), (3, 128, 64, 14, 150),
                                                (8, 64, 16, 11, 130), (4, 64, 64, 40, 33)])
def test_more_items_than_the_grid_holds(dev, window_path, path, G, D, bs, seqs, tokens):
    """Several items one after the other on each CTA pair: phases, Q and O handed on between them, and
    items that are not there in between (8 kv heads, sequences of 0 to ``tokens`` tokens)."""
    window_path(path)
    new = [tokens * (i % 5) // 4 for i in range(seqs)]
    lens = [n + 37 * (i % 4) for i, n in enumerate(new)]
    _run_prefill(dev, "bf16", 8, G, D, bs, lens, new, 64, 3, True, seed=8)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64)])
def test_empty_loose_and_padded_on_tcgen05(dev, window_path, dtype, D):
    """Sequences without new tokens, a bound above every length, rows of q and out behind the last
    sequence, which stay as they were."""
    window_path(TCGEN05)
    base.test_window_prefill_empty_and_loose(dev, dtype, D)
    c = Case(dev, dtype, 2, 4, D, 16, [50, 0, 77, 140], [50, 0, 0, 9], seed=5)
    want = _prefill(c, 40, 2)
    real = c.q
    c.q = torch.cat([real, torch.full_like(real, float("nan"))])
    got = _prefill(c, 40, 2, 300)
    assert torch.equal(got[:len(real)], want) and bool((got[len(real):] == 7.0).all())


@pytest.mark.parametrize("D", [128, 64])
def test_bad_sequences_on_tcgen05(dev, window_path, D):
    window_path(TCGEN05)
    base.test_bad_sequences(dev, "prefill", "bf16", D)


def test_bad_cu_q_on_tcgen05(dev, window_path):
    window_path(TCGEN05)
    base.test_bad_cu_q(dev)


def test_capture_on_tcgen05(dev, window_path):
    window_path(TCGEN05)
    base.test_capture_streams_and_two_calls_at_once(dev)


# ---- trees: the documented rounding of a weight ------------------------------------------

@pytest.mark.parametrize("dtype,H,G,D,bs,lens,new,window,sink", base.TREES)
def test_tree_weights(dev, dtype, H, G, D, bs, lens, new, window, sink):
    c = Case(dev, dtype, H, G, D, bs, lens, new, 16)
    kv = c.values(c.k), c.values(c.v)
    made = [_random_tree(c.rng, int(n)) for n in new]
    mask, pos = _tree_args(c, [t for t, _ in made], [d for _, d in made], -(-max(new) // 64))

    def seen_of(b, i):
        ctx = int(c.lens[b] - c.new[b])
        return MK.tree_seen(ctx, made[b][0], i, ctx + int(made[b][1][i]), window, sink)

    _check_weights(c, _tree(c, mask, pos, window, sink), *kv, seen_of, _weight(dtype, max(new) * G > 16))


# ---- a chain, and the mask that says the same ---------------------------------------------

@pytest.mark.parametrize("dtype,G,D,n", [("bf16", 4, 128, 40), ("bf16", 4, 128, 4), ("bf16", 2, 128, 100),
                                         ("bf16", 4, 64, 20), ("f32", 3, 64, 30), ("i8", 4, 128, 24)])
@pytest.mark.parametrize("window,sink,ctx", [(0, 0, 90), (3, 0, 90), (9, 2, 90), (9, 100, 90), (3, 4, 2), (5, 0, 0)])
def test_a_chain_as_a_mask(dev, dtype, G, D, n, window, sink, ctx):
    """The bits alone decide among drafted tokens, so a window layer's mask leaves out those that the
    window has passed: with such bits a chain gives what it gives without a mask, to the bit."""
    c = Case(dev, dtype, 2, G, D, 16, [ctx + n, 70], [n, 3], seed=81)
    kv = c.values(c.k), c.values(c.v)

    def seen_of(b, i):
        return MK.window_seen(int(c.lens[b] - c.new[b]) + i, window, sink)

    sees = []
    for b in range(2):
        m, at = int(c.new[b]), int(c.lens[b] - c.new[b])
        s = np.zeros((m, m), bool)
        for i in range(m):
            s[i, :i + 1] = seen_of(b, i)[at:]
        sees.append(s)
    mask, pos = _tree_args(c, sees, [np.arange(n), np.arange(3)], -(-n // 64))
    chain = _tree(c, None, None, window, sink)
    assert torch.equal(_tree(c, mask, pos, window, sink), chain)
    assert torch.equal(_tree(c, mask, None, window, sink), chain)
    _check_weights(c, chain, *kv, seen_of, _weight(dtype, n * G > 16))


# ---- one call beside others -----------------------------------------------------------------

def _jobs(dev):
    """Calls of every kernel, with shapes of their own: name -> function that gives new outputs."""
    jobs = {}
    for i, (dtype, H, G, D, lens, new) in enumerate([
            ("bf16", 2, 4, 128, [900, 70], [30, 3]), ("bf16", 8, 4, 128, [500] * 20, [300] * 20),
            ("f32", 2, 3, 64, [700], [9]), ("i8", 4, 2, 128, [300] * 20, [12] * 20),
            ("bf16", 1, 16, 64, [3000], [5]), ("bf16", 4, 2, 128, [1000, 800], [130, 64]), ("i8", 1, 12, 64, [800], [50])]):
        c = Case(dev, dtype, H, G, D, 16, lens, new, seed=91 + i)
        w = Case(dev, dtype, H, G, D, 16, lens, [1] * len(lens), seed=111 + i)
        ws, (bt, l, o, cu) = _workspace(c, max(new)), c.device()
        wbt, wl, wo, _ = w.device()
        count = _t([min(2, n) for n in new], dev)
        path = _t([[0, n - 1] for n in new], dev)

        def work(c=c, w=w, most=max(new), ws=ws, bt=bt, l=l, o=o, cu=cu, wbt=wbt, wl=wl, wo=wo, count=count, path=path):
            outs = [torch.full_like(c.q, 7.0), torch.full_like(c.q, 7.0), torch.full_like(w.q, 7.0)]
            pkv.prefill_attention_window(c.pool, c.layer, c.q, c.scale, bt, l, o, cu, most, 100, outs[0], sink=2)
            pkv.decode_attention_tree(c.pool, c.layer, c.q, c.scale, bt, l, o, cu, most, None, outs[1], ws, window=400)
            pkv.decode_attention_window(w.pool, w.layer, w.q, w.scale, wbt, wl, wo, 400, outs[2], sink=2)
            pkv.accept_tokens(c.pool, 0, bt, l, o, cu, path, count)  # (a layer that no call above reads)
            return outs

        jobs[f"{dtype} {G} {D} {i}"] = work
    return jobs


def test_calls_of_several_threads(dev):
    """Every thread's calls, on its own stream, give what they give alone, to the bit."""
    jobs = list(_jobs(dev).values())
    torch.cuda.synchronize()
    alone = [[x.clone() for x in work()] for work in jobs]
    torch.cuda.synchronize()
    bad = []

    def run(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(8):
                    got = jobs[i]()
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


def test_the_same_bits_every_time(dev):
    for name, work in _jobs(dev).items():
        first = [x.clone() for x in work()]
        for _ in range(5):
            assert all(torch.equal(a, b) for a, b in zip(first, work())), name


_CAPTURE = """
import torch
import paged_kv_cache_blk_gb300 as pkv
dev = torch.device("cuda", 0)
torch.manual_seed(1)
pkv.set_debug_window_path({path})
N, bs, H, D, G, n = 64, 16, 2, {D}, 4, {n}
kind = torch.bfloat16 if {path} else torch.float32
k = torch.randn(N, 1, bs, H, D, device=dev).to(kind)
v = torch.randn_like(k)
pool = pkv.Pool(k, v)
i = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
bt = torch.randperm(N, device=dev).int()[:40].reshape(1, 40).contiguous()
ln, cu = i([600]), torch.tensor([0, n], device=dev)
q = torch.randn(n, H * G, D, device=dev).to(kind)
one = q[:1].clone()
outs = [torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(one)]
path, count = i([list(range(1, 4))]), i([3])
ws = torch.empty(1 << 27, dtype=torch.uint8, device=dev)

def step():
    pkv.prefill_attention_window(pool, 0, q, 0.1, bt, ln, None, cu, n, 100, outs[0], sink=1)
    pkv.decode_attention_tree(pool, 0, q, 0.1, bt, ln, None, cu, n, None, outs[1], ws)
    pkv.decode_attention_window(pool, 0, one, 0.1, bt, ln, None, 100, outs[2], sink=1)
    pkv.accept_tokens(pool, 0, bt, ln, None, cu, path, count)

k0, v0 = k.clone(), v.clone()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    step()
assert torch.equal(k, k0) and not outs[0].any()
g.replay()
torch.cuda.synchronize()
a = [x.clone() for x in (*outs, k, v)]
assert all(bool(x.any()) for x in outs) and not torch.equal(k, k0)
k.copy_(k0)
v.copy_(v0)
step()
torch.cuda.synchronize()
assert all(torch.equal(x, y) for x, y in zip(a, (*outs, k, v)))
assert pkv.device_error() == "PKV_OK"
"""


@pytest.mark.parametrize("path,D,n", [(2, 128, 40), (2, 64, 40), (1, 128, 4), (0, 64, 10)])
def test_first_calls_of_a_process_inside_a_capture(dev, path, D, n):
    r = subprocess.run([sys.executable, "-c", _CAPTURE.format(path=path, D=D, n=n)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]


# ---- far places -------------------------------------------------------------------------------

FAR = [("bf16", 128, 40, TCGEN05), ("bf16", 64, 100, TCGEN05), ("bf16", 128, 3, MMA), ("f32", 64, 5, MMA),
       ("i8", 128, 9, MMA)]


def _all_calls(pool, layer, q, scale, bt, lens, cu, n, ws, window):
    """The four calls on one sequence; the outputs, and where the accepted rows went."""
    outs = [torch.full_like(q, 7.0), torch.full_like(q, 7.0), torch.full_like(q[:1], 7.0)]
    pkv.prefill_attention_window(pool, layer, q, scale, bt, lens, None, cu, n, window, outs[0])
    pkv.decode_attention_tree(pool, layer, q, scale, bt, lens, None, cu, n, None, outs[1], ws, window=window)
    pkv.decode_attention_window(pool, layer, q[-1:].contiguous(), scale, bt, lens, None, window, outs[2])
    path = _t([[1, n - 1]], q.device)
    pkv.accept_tokens(pool, layer, bt, lens, None, cu, path, _t([2], q.device))
    assert pkv.device_error() == "PKV_OK"
    return outs


@pytest.mark.parametrize("dtype,D,n,path", FAR)
def test_positions_near_two_to_the_thirty(dev, window_path, dtype, D, n, path):
    """The last rows that a table of 2^30 can name give what a short table of the same blocks gives."""
    window_path(path)
    bs = 64
    c = Case(dev, dtype, 2, 4, D, bs, [10 * bs], [n], seed=121, offsets=False)
    MB = (1 << 30) // bs
    far = torch.full((1, MB), -1, dtype=torch.int32, device=dev)
    near = _t(c.table[:, :10], dev)
    far[:, -10:] = near
    ws, cu = _workspace(c, n), _t([0, n], dev, torch.int64)
    k, v, got = c.k.clone(), c.v.clone(), []
    for bt, length in ((near, 10 * bs), (far, 1 << 30)):
        c.k.copy_(k)
        c.v.copy_(v)
        outs = _all_calls(c.pool, c.layer, c.q, c.scale, bt, _t([length], dev), cu, n, ws, 400)
        got.append(outs + [c.k.clone(), c.v.clone()])
    assert all(torch.equal(a, b) for a, b in zip(*got)) and not torch.equal(got[0][3], k)


@pytest.mark.parametrize("dtype,D,n,path", FAR)
def test_pools_past_two_to_the_32_bytes(dev, window_path, dtype, D, n, path):
    """Blocks that lie beyond 2^32 bytes of a pool give what a small pool gives."""
    window_path(path)
    H, bs, L = 8, 16, 2
    c = Case(dev, dtype, H, 4, D, bs, [9 * bs], [n], seed=131, offsets=False, layers=L)
    per_block = c.k[0].numel() * c.k.element_size()
    N = (5 << 30) // per_block + 40 if dtype != "i8" else (9 << 29) // per_block + 40
    big = [torch.empty((N,) + tuple(c.k.shape[1:]), dtype=c.k.dtype, device=dev) for _ in range(2)]
    m = c.spec.num_blocks
    for b, x in zip(big, (c.k, c.v)):
        b[N - m:] = x
    pool = pkv.Pool(*big, H, D) if dtype == "i8" else pkv.Pool(*big)
    near = _t(c.table[:, :9], dev)
    ws, cu, lens = _workspace(c, n), _t([0, n], dev, torch.int64), _t([9 * bs], dev)
    got = []
    for p, bt in ((c.pool, near), (pool, near + (N - m))):
        outs = _all_calls(p, 1, c.q, c.scale, bt, lens, cu, n, ws, 100)
        got.append(outs)
    assert all(torch.equal(a, b) for a, b in zip(*got))
    for b, x in zip(big, (c.k, c.v)):
        assert torch.equal(b[N - m:], x)


# ---- shapes that the lists above leave out ---------------------------------------------------

@pytest.mark.parametrize("dtype,H,G,D,bs,lens,new", [
    ("bf16", 1, 2, 128, 16, [900, 333], [300, 333]), ("bf16", 1, 3, 64, 32, [1400], [700]),
    ("f32", 1, 1, 64, 16, [500, 300], [257, 300]), ("i8", 1, 2, 128, 16, [700], [400]),
    ("bf16", 105, 1, 64, 16, [300, 40], [40, 3]), ("bf16", 33, 2, 128, 8, [200], [20])])
def test_wide_trees_and_many_heads(dev, dtype, H, G, D, bs, lens, new):
    """Masks of several words over several units, and kv heads of any number."""
    c = Case(dev, dtype, H, G, D, bs, lens, new, 151)
    kv = c.values(c.k), c.values(c.v)
    made = [_random_tree(c.rng, int(n)) for n in new]
    words = -(-max(new) // 64) + 1
    mask, pos = _tree_args(c, [t for t, _ in made], [d for _, d in made], words)

    def seen_of(b, i):
        ctx = int(c.lens[b] - c.new[b])
        return MK.tree_seen(ctx, made[b][0], i, ctx + int(made[b][1][i]), 90, 5)

    _check_weights(c, _tree(c, mask, pos, 90, 5), *kv, seen_of, _weight(dtype, max(new) * G > 16))


@pytest.mark.parametrize("dtype,D,n", [("bf16", 128, 3), ("bf16", 128, 20), ("bf16", 128, 100), ("bf16", 64, 20),
                                       ("f32", 64, 9), ("i8", 128, 12)])
def test_rows_behind_the_last_sequence_stay(dev, window_path, dtype, D, n):
    """A padded batch: more rows of q (NaN), out, mask and positions than cu_q names, and a bound above
    every length.  (The bound chooses the kernel and the split: to rounding, tests above hold the rest.)"""
    c = Case(dev, dtype, 2, 4, D, 16, [90 + n, 40, n], [n, 0, n], seed=161)
    made = [_random_tree(c.rng, int(m)) for m in c.new]
    mask, pos = _tree_args(c, [t for t, _ in made], [d for _, d in made], 4)
    real = c.q
    want = {"tree": _tree(c, mask, pos, most=150), "chain": _tree(c, None, None, most=150), "prefill": _prefill(c, 40, 2, 150)}
    pad = lambda x, v: torch.cat([x, torch.full((33,) + tuple(x.shape[1:]), v, dtype=x.dtype, device=dev)])
    c.q = pad(real, float("nan"))
    got = {"tree": _tree(c, pad(mask, -1), pad(pos, -1), most=150), "chain": _tree(c, None, None, most=150),
           "prefill": _prefill(c, 40, 2, 150)}
    for k, x in got.items():
        assert torch.equal(x[:len(real)], want[k]) and bool((x[len(real):] == 7.0).all()), k
    assert pkv.device_error() == "PKV_OK"


def test_one_workspace_for_calls_in_a_row(dev):
    """Calls on one stream may share a workspace, of any size that the largest asks for."""
    cases = [Case(dev, "bf16", 2, 4, 128, 16, [700, 90], [m, 2], seed=171 + m) for m in (3, 40, 12, 100, 4)]
    big = torch.full((max(_workspace(c, int(c.new.max())).numel() for c in cases),), 255, dtype=torch.uint8, device=dev)
    want = [_tree(c, None, None) for c in cases]
    args = [c.device() for c in cases]
    outs = [torch.full_like(c.q, 7.0) for c in cases]
    torch.cuda.synchronize()
    for c, (bt, lens, offs, cu), out in zip(cases, args, outs):
        pkv.decode_attention_tree(c.pool, c.layer, c.q, c.scale, bt, lens, offs, cu, int(c.new.max()), None, out, big)
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
