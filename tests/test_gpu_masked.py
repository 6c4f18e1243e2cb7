"""GPU parity of windowed decode and prefill attention, tree verification and the
moves of accepted tokens, against the oracle.

Tolerances.  For a result o = sum w_i v_i, with A = sum w_i |v_i| and X = scale *
max_i sum_d |q_d k_id|: an error of d in a score changes its weight by the factor
e^d, and o by 2 d A at most.
* Scores, bf16 and int8: products exact, at most D + 8 sums in fp32, truncated on the
  tensor cores: d <= (D + 8) 2^-23 X, and 2^-21 for the exponential.
  fp32: each product of two tf32 pairs within 3 * 2^-22, 3 D / 8 + 2 sums: d <=
  (3 D / 8 + 8) 2^-23 X + 2^-21 (the FMA form of the single-token call: D + 8 sums).
* P V: n sums in fp32, n 2^-23 A.  The weight's own rounding: two bf16 parts 2^-16 A
  (fp16 parts: less, and 2^-27 of the largest), one bf16 part (more than 16
  rows a kv head) 2^-8 A; tf32 3 * 2^-22 A.
* The output's rounding: half a step, 2^-8 |o| (bf16), 2^-24 |o| (fp32), of a value
  that the errors above may have moved to the next binade (1.01).
"""

import numpy as np
import pytest
import torch

import paged_kv_cache_blk_gb300 as pkv
from oracle import masked as MK
from oracle import quant as Q
from paged_kv_cache_blk_gb300 import PkvError
from workloads import PoolSpec, rand_rows, to_numpy_bits
from workloads.gen import fill_pool_i8

from gpu_util import need_gpu, widen_out

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    d = need_gpu()
    pkv.set_validate(False)
    pkv.device_error(clear=True)
    return d


def _t(a, dev, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev, dtype)


def _io(dtype):
    return "f32" if dtype == "f32" else "bf16"


class Case:
    """A pool, ragged sequences in it and their new tokens."""

    def __init__(self, dev, dtype, H, G, D, bs, lens, new, seed=3, layers=2, offsets=True,
                 extra_blocks=0):
        rng = np.random.default_rng(seed)
        self.rng, self.dev, self.dtype, self.seed = rng, dev, dtype, seed
        self.H, self.G, self.D, self.bs, self.layer = H, G, D, bs, layers - 1
        self.lens, self.new = np.asarray(lens, np.int64), np.asarray(new, np.int64)
        B = len(lens)
        self.offs = rng.integers(0, bs, B) if offsets else np.zeros(B, np.int64)
        nblk = -(-(self.offs + self.lens) // bs)
        N = int(nblk.sum()) + 2
        ids, at = rng.permutation(N), 0
        self.table = np.full((B, max(1, int(nblk.max())) + extra_blocks), -1, np.int64)
        for b in range(B):
            self.table[b, :nblk[b]] = ids[at:at + nblk[b]]
            at += nblk[b]
        self.home = self.table.copy()  # (poison() writes to table)
        self.cu = np.concatenate([[0], np.cumsum(self.new)])
        self.spec = PoolSpec(N, layers, bs, H, D, dtype)
        if dtype == "i8":
            self.k = torch.zeros(self.spec.shape, dtype=torch.uint8, device=dev)
            self.v = torch.zeros_like(self.k)
            for l in range(layers):
                fill_pool_i8(self.k, self.v, self.spec, l, seed + l)
            self.pool = pkv.Pool(self.k, self.v, H, D)
        else:
            self.k = rand_rows(self.spec.shape, dtype, seed + 1, dev)
            self.v = rand_rows(self.spec.shape, dtype, seed + 2, dev)
            self.pool = pkv.Pool(self.k, self.v)
        self.q = rand_rows((int(self.cu[-1]), H * G, D), _io(dtype), seed + 3, dev)
        self.scale = D ** -0.5

    def values(self, cache):
        """The layer in 64 bits, [blocks, bs, H, D]."""
        if self.dtype != "i8":
            return widen_out(cache[:, self.layer])
        rows = to_numpy_bits(cache[:, self.layer].contiguous()).reshape(-1, self.spec.row_bytes)
        codes, scales = Q.unpack_rows(rows, self.H, self.D)
        x = codes.astype(np.float64) * scales[..., None].astype(np.float64)
        return x.reshape(self.spec.num_blocks, self.bs, self.H, self.D)

    def rows(self, b):
        """Table blocks and rows of the positions of a sequence."""
        p = self.offs[b] + np.arange(self.lens[b])
        return self.home[b, p // self.bs], p % self.bs

    def device(self):
        return (_t(self.table, self.dev), _t(self.lens, self.dev), _t(self.offs, self.dev),
                _t(self.cu, self.dev, torch.int64))

    def poison(self, seen):
        """``seen``: per sequence, which keys some query sees.  The others hold NaN (an int8 pool:
        scales of NaN), as do rows outside the sequences and other layers; table entries without
        a seen key are out of range."""
        live = np.zeros((self.spec.num_blocks, self.spec.num_layers, self.bs), bool)
        for b in range(len(self.lens)):
            blk, row = self.rows(b)
            live[blk[seen[b]], self.layer, row[seen[b]]] = True
            used = np.unique((self.offs[b] + np.flatnonzero(seen[b])) // self.bs)
            dead = np.setdiff1d(np.arange(self.table.shape[1]), used)
            self.table[b, dead] = np.where(np.arange(len(dead)) % 2, -1, 1 << 29)
        dead = _t(~live, self.dev, torch.bool)
        for c in (self.k, self.v):
            if self.dtype == "i8":
                c[..., self.H * self.D:self.H * self.D + 4 * self.H].view(torch.float32).masked_fill_(
                    dead[..., None], float("nan"))
            else:
                c.masked_fill_(dead[..., None, None], float("nan"))

    def check(self, got, kvals, vvals, seen_of, weight_err, fma=False):
        """``seen_of(b, i)``: the keys that new token i of sequence b sees."""
        D, G = self.D, self.G
        got, q = widen_out(got), widen_out(self.q)
        bf16 = self.dtype != "f32"
        for b in range(len(self.lens)):
            blk, row = self.rows(b)
            for g in range(self.H):
                k, v = kvals[blk, row, g], vvals[blk, row, g]
                for i in range(int(self.new[b])):
                    t, seen = int(self.cu[b]) + i, seen_of(b, i)
                    full = np.zeros(len(k), bool)
                    full[:len(seen)] = seen
                    ref, mean, top = MK.attention(q[t, g * G:(g + 1) * G], k, v, full, self.scale)
                    x = abs(self.scale) * top[:, None]
                    sums = D + 8 if bf16 or fma else 3 * D // 8 + 8
                    d = sums * 2.0 ** -23 * x + 2.0 ** -21
                    n = int(full.sum())
                    tol = (2 * d + n * 2.0 ** -23 + weight_err) * mean
                    if self.dtype == "i8" and fma:  # (two fp16 parts, of the largest product)
                        tol += n * 2.0 ** -27 * (np.abs(v[full]).max() if n else 0)
                    tol += np.abs(ref) * 1.01 * (2.0 ** -8 if bf16 else 2.0 ** -24)
                    err = np.abs(got[t, g * G:(g + 1) * G] - ref)
                    assert np.all(err <= tol + 1e-30), (b, i, g, float((err - tol).max()), float(err.max()))
        assert pkv.device_error() == "PKV_OK"


def _weight_err(dtype, one_part=False):
    if dtype == "f32":
        return 3 * 2.0 ** -22
    return 2.0 ** -8 if one_part else 2.0 ** -16


# ---- windowed decode --------------------------------------------------------------

def _window(c, window, sink, out=None):
    bt, lens, offs, _ = c.device()
    out = torch.full_like(c.q, 7.0) if out is None else out
    pkv.decode_attention_window(c.pool, c.layer, c.q, c.scale, bt, lens, offs, window, out, sink=sink)
    return out


def _run_window(dev, dtype, H, G, D, bs, lens, window, sink, seed=3, poison=True, extra=0):
    c = Case(dev, dtype, H, G, D, bs, lens, np.ones(len(lens), np.int64), seed, extra_blocks=extra)
    kv = c.values(c.k), c.values(c.v)
    seen = [MK.window_seen(n - 1, window, sink) if n else np.zeros(0, bool) for n in lens]
    if poison:
        c.poison(seen)
    c.check(_window(c, window, sink), *kv, lambda b, i: seen[b], _weight_err(dtype), fma=True)


WINDOWS = [
    ("bf16", 8, 4, 128, 16, [300, 1, 16, 17, 0, 131], 32, 4), ("bf16", 2, 1, 64, 8, [200, 3], 1, 0),
    ("bf16", 1, 16, 128, 16, [500], 333, 17), ("bf16", 3, 9, 64, 1, [40, 9], 7, 2),
    ("bf16", 2, 3, 128, 64, [700, 64], 65, 70), ("bf16", 1, 8, 64, 1024, [2100, 1500], 1200, 3),
    ("f32", 4, 3, 64, 32, [300, 1, 90], 40, 33), ("f32", 2, 1, 128, 16, [260], 16, 1),
    ("f32", 1, 16, 128, 8, [100, 50], 49, 8), ("f32", 3, 5, 64, 2, [60], 9, 5),
    ("i8", 8, 4, 128, 16, [300, 1, 17, 0], 40, 4), ("i8", 2, 16, 64, 8, [120], 31, 0),
    ("i8", 3, 1, 64, 16, [99, 33], 33, 1), ("i8", 5, 2, 128, 1, [30], 3, 1),
]


@pytest.mark.parametrize("dtype,H,G,D,bs,lens,window,sink", WINDOWS)
def test_window_decode(dev, dtype, H, G, D, bs, lens, window, sink):
    _run_window(dev, dtype, H, G, D, bs, lens, window, sink)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "i8"])
@pytest.mark.parametrize("D", [64, 128])
def test_window_decode_long(dev, dtype, D):
    """Windows over many tiles, on clusters of CTAs, and over whole sequences."""
    _run_window(dev, dtype, 2, 4, D, 16, [30000, 5000], 9000, 100, seed=11)
    _run_window(dev, dtype, 1, 2, D, 16, [4000], 2 ** 31 - 1, 2 ** 31 - 1, seed=12, extra=3)
    _run_window(dev, dtype, 8, 2, D, 16, [300 + 7 * i for i in range(60)], 128, 4, seed=13)


def test_window_of_everything_is_decode_attention(dev):
    """A window over the whole sequence gives what decode_attention_sparse gives over all blocks,
    to the bit."""
    c = Case(dev, "bf16", 2, 4, 128, 16, [700, 33, 5], [1, 1, 1])
    bt, lens, offs, _ = c.device()
    a = _window(c, 700, 0)
    mb = c.table.shape[1]
    sel = torch.arange(mb, device=dev, dtype=torch.int32).expand(3, 2, mb).contiguous()
    out = torch.empty_like(a)
    pkv.decode_attention_sparse(c.pool, c.layer, c.q, c.scale, bt, offs,
                                torch.arange(3, device=dev, dtype=torch.int32), lens - 1, sel, out)
    assert torch.equal(a, out)


# ---- windowed prefill -------------------------------------------------------------

def _prefill(c, window, sink, most=None, out=None):
    bt, lens, offs, cu = c.device()
    out = torch.full_like(c.q, 7.0) if out is None else out
    pkv.prefill_attention_window(c.pool, c.layer, c.q, c.scale, bt, lens, offs, cu,
                                 int(c.new.max()) if most is None else most, window, out, sink=sink)
    return out


def _run_prefill(dev, dtype, H, G, D, bs, lens, new, window, sink, seed=4, most=None):
    c = Case(dev, dtype, H, G, D, bs, lens, new, seed, extra_blocks=seed % 3)
    kv = c.values(c.k), c.values(c.v)

    def seen_of(b, i):
        return MK.window_seen(int(c.lens[b] - c.new[b]) + i, window, sink)

    some = []
    for b in range(len(lens)):
        s = np.zeros(int(c.lens[b]), bool)
        for i in range(int(c.new[b])):
            x = seen_of(b, i)
            s[:len(x)] |= x
        some.append(s)
    c.poison(some)
    got = _prefill(c, window, sink, most)
    rows = (max(new) if most is None else most) * G
    c.check(got, *kv, seen_of, _weight_err(dtype, rows > 16))


PREFILLS = [
    ("bf16", 2, 4, 128, 16, [100], [100], 30, 4), ("bf16", 2, 4, 128, 16, [300, 37, 129], [300, 37, 129], 64, 0),
    ("bf16", 2, 4, 128, 16, [700, 260], [40, 260], 129, 5), ("bf16", 1, 1, 128, 16, [400, 130], [400, 5], 100, 1),
    ("bf16", 2, 2, 128, 32, [333, 64], [100, 64], 1, 0), ("bf16", 1, 8, 128, 16, [400, 17], [33, 17], 200, 150),
    ("bf16", 1, 16, 128, 8, [150, 90], [150, 8], 17, 3), ("bf16", 1, 4, 128, 128, [900, 1], [300, 1], 300, 2),
    ("bf16", 2, 4, 128, 64, [1000, 520, 33, 95], [1000, 520, 33, 95], 257, 40),
    ("bf16", 2, 4, 64, 16, [700, 260, 33], [700, 40, 33], 129, 5), ("bf16", 1, 8, 64, 64, [900, 70], [300, 70], 300, 2),
    ("bf16", 1, 1, 64, 8, [500], [400], 90, 17), ("bf16", 1, 16, 64, 32, [300], [150], 1, 0),
    ("bf16", 1, 2, 64, 128, [400], [200], 130, 4), ("bf16", 2, 3, 128, 16, [700, 129], [600, 129], 200, 9),
    ("bf16", 1, 5, 128, 64, [500], [300], 64, 1), ("bf16", 1, 7, 64, 16, [400, 90], [400, 33], 150, 2),
    ("bf16", 1, 11, 128, 8, [250], [100], 33, 1), ("bf16", 1, 13, 64, 32, [200], [200], 70, 0),
    ("bf16", 1, 4, 128, 16, [1500], [700], 5000, 9),
    ("bf16", 2, 3, 128, 16, [150, 20], [150, 3], 50, 4), ("bf16", 1, 5, 64, 16, [200, 70], [130, 70], 64, 1),
    ("bf16", 2, 1, 64, 4, [90], [90], 20, 2), ("bf16", 1, 2, 128, 256, [600], [300], 280, 10),
    ("bf16", 1, 2, 128, 1, [80], [30], 9, 3), ("bf16", 1, 16, 64, 1024, [1300], [40], 1100, 1),
    ("f32", 2, 3, 64, 32, [300, 1, 90], [300, 1, 40], 70, 1), ("f32", 1, 4, 128, 16, [130], [90], 33, 5),
    ("f32", 1, 1, 64, 8, [70], [70], 1, 1), ("f32", 1, 9, 128, 2, [50], [20], 25, 0),
    ("i8", 2, 4, 128, 16, [260, 31], [260, 31], 100, 4), ("i8", 3, 1, 64, 8, [120], [64], 50, 7),
    ("i8", 1, 12, 128, 64, [200], [30], 90, 100), ("i8", 5, 2, 64, 1, [40], [40], 10, 0),
]


@pytest.mark.parametrize("dtype,H,G,D,bs,lens,new,window,sink", PREFILLS)
def test_window_prefill(dev, dtype, H, G, D, bs, lens, new, window, sink):
    _run_prefill(dev, dtype, H, G, D, bs, lens, new, window, sink)


@pytest.mark.parametrize("dtype,H,G,D,bs,lens,new,window,sink", [
    ("i8", 2, 2, 128, 8, [5000, 300, 2], [3, 3, 2], 2166, 4), ("bf16", 1, 4, 64, 16, [3000], [4], 2000, 0),
    ("bf16", 8, 4, 128, 16, [2500, 900], [4, 1], 2000, 9), ("bf16", 1, 16, 128, 32, [4000], [4], 3000, 1),
    ("f32", 2, 3, 64, 16, [1500, 40], [5, 5], 1000, 2), ("f32", 1, 8, 128, 4, [700], [3], 600, 40),
    ("i8", 1, 8, 64, 2, [900], [4], 800, 1), ("f32", 1, 8, 128, 16, [900], [8], 700, 1),
    ("bf16", 1, 2, 64, 16, [900], [300], 400, 3),
])
def test_window_prefill_of_few_tokens(dev, dtype, H, G, D, bs, lens, new, window, sink):
    """Few rows under a long window: their keys shared out over a cluster of CTAs."""
    _run_prefill(dev, dtype, H, G, D, bs, lens, new, window, sink, seed=15)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("i8", 128), ("f32", 64)])
def test_window_prefill_empty_and_loose(dev, dtype, D):
    """Sequences without new tokens between others, a bound above every length."""
    _run_prefill(dev, dtype, 2, 4, D, 16, [50, 0, 77, 140], [50, 0, 0, 9], 40, 2, seed=5, most=500)


# ---- trees ------------------------------------------------------------------------

def _random_tree(rng, n):
    sees = np.zeros((n, n), bool)
    depth = np.zeros(n, np.int64)
    for i in range(n):
        parent = int(rng.integers(-1, i)) if i else -1
        if parent >= 0:
            sees[i] = sees[parent]
            depth[i] = depth[parent] + 1
        sees[i, i] = True
    return sees, depth


def _tree_args(c, trees, depths, words):
    mask = np.zeros((int(c.cu[-1]), words), np.uint64)
    pos = np.zeros(int(c.cu[-1]), np.int64)
    for b, sees in enumerate(trees):
        mask[c.cu[b]:c.cu[b + 1]] = MK.mask_words(sees, words)
        pos[c.cu[b]:c.cu[b + 1]] = c.lens[b] - c.new[b] + depths[b]
    return _t(mask.view(np.int64), c.dev, torch.int64), _t(pos, c.dev)


def _workspace(c, most, fill=255):
    n = pkv.decode_tree_workspace_size(c.pool, len(c.lens), c.H * c.G, most)
    return torch.full((n,), fill, dtype=torch.uint8, device=c.dev)  # (NaN, read as floats)


def _tree(c, mask, pos, window=0, sink=0, most=None, out=None):
    bt, lens, offs, cu = c.device()
    out = torch.full_like(c.q, 7.0) if out is None else out
    most = max(1, int(c.new.max())) if most is None else most
    pkv.decode_attention_tree(c.pool, c.layer, c.q, c.scale, bt, lens, offs, cu, most, mask, out,
                              _workspace(c, most), q_pos=pos, window=window, sink=sink)
    return out


def _run_tree(dev, dtype, H, G, D, bs, lens, new, window, sink, words=None, seed=6, trees=None,
              chain=False, most=None, use_pos=True):
    c = Case(dev, dtype, H, G, D, bs, lens, new, seed, extra_blocks=seed % 3)
    kv = c.values(c.k), c.values(c.v)
    made = [_random_tree(c.rng, int(n)) for n in new]
    sees, depth = [t for t, _ in made], [d for _, d in made]
    if trees is not None:
        sees = trees
    words = words or -(-int(max(new)) // 64)

    def seen_of(b, i):
        ctx = int(c.lens[b] - c.new[b])
        if chain:
            return MK.window_seen(ctx + i, window, sink)
        pos = ctx + (int(depth[b][i]) if use_pos else i)
        return MK.tree_seen(ctx, sees[b][:, :int(new[b])], i, pos, window, sink)

    some = []
    for b in range(len(lens)):
        s = np.zeros(int(c.lens[b]), bool)
        for i in range(int(new[b])):
            x = seen_of(b, i)
            s[:len(x)] |= x
        if new[b]:
            s[int(c.lens[b] - c.new[b]):] = True  # drafted rows are stored, seen or not
        some.append(s)
    c.poison(some)
    mask, pos = (None, None) if chain else _tree_args(c, sees, depth, words)
    got = _tree(c, mask, pos if use_pos else None, window, sink, most)
    c.check(got, *kv, seen_of, _weight_err(dtype, max(new if most is None else [most]) * G > 16))


TREES = [
    ("bf16", 2, 4, 128, 16, [300, 40, 9], [3, 2, 4], 0, 0), ("bf16", 2, 4, 128, 16, [500, 77], [8, 5], 0, 0),
    ("bf16", 2, 4, 128, 16, [900, 64, 400], [64, 64, 11], 0, 0), ("bf16", 1, 1, 128, 16, [333], [17], 0, 0),
    ("bf16", 1, 1, 128, 8, [1500, 140], [130, 129], 0, 0), ("bf16", 1, 8, 128, 64, [700, 65], [33, 20], 0, 0),
    ("bf16", 1, 16, 128, 128, [600], [40], 0, 0), ("bf16", 2, 2, 128, 32, [2000, 1000], [100, 64], 130, 5),
    ("bf16", 2, 4, 128, 16, [900, 300], [64, 20], 300, 4), ("bf16", 1, 16, 128, 16, [400, 30], [16, 16], 40, 0),
    ("bf16", 2, 4, 64, 16, [900, 64, 400], [64, 64, 11], 0, 0), ("bf16", 1, 1, 64, 8, [1500, 140], [130, 129], 200, 3),
    ("bf16", 1, 16, 64, 128, [600, 90], [40, 7], 0, 0), ("bf16", 2, 8, 64, 32, [500], [16], 100, 4),
    ("bf16", 1, 3, 128, 16, [900, 300], [84, 85], 0, 0), ("bf16", 2, 5, 128, 64, [400, 50], [26, 50], 77, 1),
    ("bf16", 1, 7, 64, 16, [700], [100], 0, 0), ("bf16", 1, 13, 128, 8, [300], [20], 0, 0),
    ("bf16", 1, 9, 64, 16, [300, 20], [14, 15], 0, 0),
    ("bf16", 2, 3, 128, 16, [200, 50], [7, 30], 0, 0), ("bf16", 3, 1, 64, 8, [120], [5], 30, 3),
    ("bf16", 1, 16, 64, 1, [90], [70], 0, 0), ("bf16", 2, 5, 64, 512, [1100, 600], [13, 4], 600, 20),
    ("f32", 2, 5, 64, 16, [300, 3], [17, 3], 0, 0), ("f32", 1, 4, 128, 16, [150, 100], [4, 1], 64, 4),
    ("f32", 2, 1, 128, 32, [400], [20], 0, 0), ("f32", 1, 16, 64, 2, [80], [9], 20, 2),
    ("f32", 1, 2, 128, 8, [200], [40], 0, 0),
    ("i8", 2, 4, 128, 16, [300, 70], [8, 3], 0, 0), ("i8", 4, 1, 64, 8, [200, 20], [12, 20], 0, 0),
    ("i8", 1, 9, 128, 32, [500], [30], 100, 10), ("i8", 3, 2, 64, 1, [60], [40], 0, 0),
    ("i8", 1, 16, 64, 128, [300], [70], 0, 0),
]


@pytest.mark.parametrize("dtype,H,G,D,bs,lens,new,window,sink", TREES)
def test_tree(dev, dtype, H, G, D, bs, lens, new, window, sink):
    _run_tree(dev, dtype, H, G, D, bs, lens, new, window, sink)


@pytest.mark.parametrize("dtype,G,D", [("bf16", 4, 128), ("bf16", 4, 64), ("f32", 3, 128), ("i8", 4, 128)])
def test_tree_chain(dev, dtype, G, D):
    """No mask: each drafted token sees those before it, under a window too."""
    _run_tree(dev, dtype, 2, G, D, 16, [400, 37, 12], [12, 37, 1], 0, 0, chain=True)
    _run_tree(dev, dtype, 2, G, D, 16, [400, 37, 12], [12, 20, 1], 9, 3, chain=True)
    _run_tree(dev, dtype, 1, G, D, 16, [70], [70], 20, 0, chain=True)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("f32", 64), ("i8", 64)])
@pytest.mark.parametrize("n", [3, 20])
def test_tree_odd_masks(dev, dtype, D, n):
    """Rows that see no drafted token, with and without a context; bits behind the last token;
    more words than are used; positions left out; a loose bound."""
    rng = np.random.default_rng(8)
    for ctx in (0, 50):
        sees = rng.random((n, n)) < 0.4
        sees[0] = False
        wide = np.zeros((n, 192), bool)
        wide[:, :n] = sees
        wide[:, n:] = rng.random((n, 192 - n)) < 0.5
        c_lens, c_new = [ctx + n, n, 64], [n, 0, 1]
        _run_tree(dev, dtype, 2, 4, D, 16, c_lens, c_new, 0, 0, words=3,
                  trees=[wide, np.zeros((0, 192), bool), np.ones((1, 192), bool)], seed=9, most=70)
        _run_tree(dev, dtype, 2, 4, D, 16, c_lens, c_new, 13, 2, words=3, use_pos=False,
                  trees=[wide, np.zeros((0, 192), bool), np.ones((1, 192), bool)], seed=9)


@pytest.mark.parametrize("dtype,D,n", [("bf16", 128, 8), ("bf16", 128, 40), ("bf16", 64, 8), ("bf16", 64, 40), ("f32", 64, 3),
                                       ("i8", 128, 16)])
def test_tree_split(dev, dtype, D, n):
    """Units split over many CTAs, units finished by one, and sequences of no tokens between."""
    _run_tree(dev, dtype, 1, 4, D, 16, [20000], [n], 0, 0, seed=10)
    if dtype == "bf16":
        _run_tree(dev, dtype, 1, 3, D, 32, [9000, 700, 50], [n, n, n], 0, 0, seed=12)
    lens = [int(x) for x in np.random.default_rng(3).integers(40, 900, 30)]
    new = [n if i % 3 else 0 for i in range(30)]
    _run_tree(dev, dtype, 2, 2, D, 16, lens, new, 0, 0, seed=11)


def test_tree_many_sequences(dev):
    """More sequences than the CTAs have threads."""
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(3, 30, 700)]
    new = [int(x) for x in rng.integers(0, 4, 700)]
    _run_tree(dev, "bf16", 1, 2, 64, 8, lens, new, 0, 0, seed=14)
    _run_tree(dev, "bf16", 1, 16, 128, 8, lens, new, 0, 0, seed=14)


@pytest.mark.parametrize("H,G,D,lens,new", [
    (8, 4, 128, [5000, 300], [4, 3]), (8, 4, 64, [2500, 900, 3], [8, 5, 3]), (3, 5, 128, [6000, 41], [12, 0]),
    (105, 1, 64, [700, 90], [3, 16]), (5, 2, 64, list(range(20, 340)), [3, 0, 2, 1] * 80)])
def test_tree_i8_heads(dev, H, G, D, lens, new):
    """Heads whose units are split in the same way, and 105 of them, which would leave CTAs idle."""
    _run_tree(dev, "i8", H, G, D, 16, lens, new, 0, 0, seed=21)


# ---- values that some queries see and others do not -------------------------------------

@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype,G,D,ctx,n", [
    ("bf16", 4, 128, 300, 40), ("bf16", 4, 128, 300, 20), ("bf16", 4, 128, 300, 6), ("bf16", 4, 128, 6000, 40),
    ("bf16", 4, 128, 6000, 20), ("bf16", 2, 64, 300, 100), ("bf16", 2, 64, 4000, 20), ("bf16", 3, 64, 700, 5),
    ("f32", 3, 64, 500, 9), ("f32", 1, 128, 2000, 30), ("i8", 4, 128, 300, 12), ("i8", 2, 64, 3000, 5)])
def test_unseen_values_do_not_spread(dev, dtype, G, D, ctx, n, bad):
    """A V row of NaN or infinities shows in the queries that see it and in no other: a drafted
    token's siblings, the tokens before it, those that its window has left behind."""
    c = Case(dev, dtype, 2, G, D, 16, [ctx + n, 70], [n, 3], seed=51)
    sees, depth = _random_tree(c.rng, n)
    mask, pos = _tree_args(c, [sees, np.tril(np.ones((3, 3)))], [depth, np.arange(3)], -(-n // 64))
    j = n // 2
    place = int(c.offs[0]) + ctx + j
    blk, row = int(c.home[0, place // 16]), place % 16
    calls = {"tree": lambda: _tree(c, mask, pos), "chain": lambda: _tree(c, None, None),
             "prefill": lambda: _prefill(c, 3, 1), "wide": lambda: _prefill(c, 1 << 20, 0)}
    seen = {"tree": sees[:, j], "chain": np.arange(n) >= j,
            "prefill": np.array([j <= i < j + 3 for i in range(n)]), "wide": np.arange(n) >= j}
    clean = {k: f() for k, f in calls.items()}
    if dtype == "i8":
        c.v[blk, c.layer, row, 2 * D:2 * D + 8].view(torch.float32).fill_(bad)
    else:
        c.v[blk, c.layer, row] = bad
    for k, f in calls.items():
        got = f()
        assert bool(got[n:].isfinite().all()), k
        touched = torch.from_numpy(seen[k]).to(dev)
        keep = got[:n][~touched].float()
        assert bool(keep.isfinite().all()), k
        # (computed another way: two roundings of the output apart, and those of the weights)
        want = clean[k][:n][~touched].float()
        assert float((keep - want).abs().max() if keep.numel() else 0.0) <= (0.04 if dtype != "f32" else 1e-5), k
        assert not bool(got[:n][touched].isfinite().any()) or dtype == "i8", k
    assert pkv.device_error() == "PKV_OK"


@pytest.mark.parametrize("D,G,n", [(64, 4, 3), (128, 4, 7), (128, 8, 8), (64, 16, 9)])
@pytest.mark.parametrize("heavy", [False, True])
def test_i8_scales_far_apart(dev, D, G, n, heavy):
    """V scales from 2^-24 to 2^24: each product counts for what it is, whether the keys of great
    scale carry weight or (``heavy`` False) next to none.  Every weight is off by 2^-11 of itself
    (one fp16) and by 2^-27 of the largest product so far, times a code of up to 127."""
    c = Case(dev, "i8", 2, G, D, 16, [150 + n, 40], [n, 2], seed=77)
    at = c.v[..., 2 * D:2 * D + 8].view(torch.float32)
    e = c.rng.integers(-24, 25, at.shape)
    e[..., 0] = np.where(c.rng.random(e.shape[:-1]) < 0.03, 24, -20)
    at.copy_(torch.from_numpy(2.0 ** e).to(dev, torch.float32))
    if not heavy:  # great V scales beside keys that point away from every query
        c.q.copy_(c.q.abs())
        big = (at[..., 0] > 1) | (at[..., 1] > 2.0 ** 10)
        c.k[..., :2 * D] = torch.where(big[..., None], torch.full_like(c.k[..., :2 * D], 28), c.k[..., :2 * D])
    k, v = c.values(c.k), c.values(c.v)
    sees, depth = _random_tree(c.rng, n)
    mask, pos = _tree_args(c, [sees, np.tril(np.ones((2, 2)))], [depth, np.arange(2)], 1)
    outs = {"tree": _tree(c, mask, pos), "prefill": _prefill(c, 90, 2)}
    q = widen_out(c.q)
    for name, out in outs.items():
        got = widen_out(out)
        for b in range(2):
            blk, row = c.rows(b)
            ctx = int(c.lens[b] - c.new[b])
            for i in range(int(c.new[b])):
                full = np.zeros(len(blk), bool)
                if name == "tree":
                    s = MK.tree_seen(ctx, sees if b == 0 else np.tril(np.ones((2, 2), bool)), i,
                                     ctx + i, 0, 0)
                else:
                    s = MK.window_seen(ctx + i, 90, 2)
                full[:len(s)] = s
                for g in range(2):
                    rows = slice(g * G, g * G + G)
                    t = int(c.cu[b]) + i
                    kk, vv = k[blk, row, g], v[blk, row, g]
                    ref, mean, top = MK.attention(q[t, rows], kk, vv, full, c.scale)
                    x = c.scale * (q[t, rows] @ kk[full].T)
                    w = np.exp(x - x.max(1, keepdims=True))
                    w /= w.sum(1, keepdims=True)
                    scales = np.abs(vv[full]).max(1) / 127
                    most = (w * scales).max(1, keepdims=True)
                    d = (D + 8) * 2.0 ** -23 * c.scale * top[:, None] + 2.0 ** -21
                    n_keys = int(full.sum())
                    tol = (2 * d + n_keys * 2.0 ** -23 + 2.0 ** -11) * mean
                    tol += n_keys * 127 * 2.0 ** -27 * most + 1.01 * 2.0 ** -8 * np.abs(ref)
                    err = np.abs(got[t, rows] - ref)
                    assert np.all(err <= tol), (name, b, i, g, float((err / tol).max()))


# ---- accepted tokens ----------------------------------------------------------------

def _accept_case(dev, dtype, H, D, bs, lens, new, paths, layers=3):
    c = Case(dev, dtype, H, 1, D, bs, lens, new, 7, layers=layers)
    most = max(1, max(len(p) for p in paths)) + 1
    table = np.full((len(paths), most), -7, np.int64)
    for b, p in enumerate(paths):
        table[b, :len(p)] = p
    return c, _t(table, dev), _t([len(p) for p in paths], dev)


def _moved(c, cache, paths, layers):
    want = cache.clone()
    for b, p in enumerate(paths):
        for src, dst in MK.accept_moves(int(c.offs[b] + c.lens[b] - c.new[b]), p):
            sb, db = int(c.table[b, src // c.bs]), int(c.table[b, dst // c.bs])
            for l in layers:
                want[db, l, dst % c.bs] = cache[sb, l, src % c.bs]
    return want


@pytest.mark.parametrize("dtype,H,D,bs", [("bf16", 8, 128, 16), ("bf16", 1, 64, 1), ("f32", 2, 64, 8),
                                          ("i8", 3, 128, 16), ("i8", 8, 64, 64), ("bf16", 1, 8, 256),
                                          ("f32", 16, 256, 16)])
@pytest.mark.parametrize("layer", [-1, 1])
def test_accept(dev, dtype, H, D, bs, layer):
    paths = [[0, 1, 2], [1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12], [], [5], [0, 2, 4, 29], list(range(1, 40))]
    new = [3, 13, 4, 6, 30, 40]
    c, table, count = _accept_case(dev, dtype, H, D, bs, [100, 13, 4, 40, 64, 90], new, paths)
    layers = range(3) if layer < 0 else [layer]
    want = [_moved(c, x, paths, layers) for x in (c.k, c.v)]
    bt, lens, offs, cu = c.device()
    pkv.accept_tokens(c.pool, layer, bt, lens, offs, cu, table, count)
    assert torch.equal(c.k, want[0]) and torch.equal(c.v, want[1])
    assert pkv.device_error() == "PKV_OK"


def test_accept_long_path(dev):
    """More tokens than one round of a CTA holds."""
    n = 2500
    path = np.sort(np.random.default_rng(2).choice(n, 2100, replace=False))
    c, table, count = _accept_case(dev, "bf16", 1, 64, 16, [n + 9], [n], [path], layers=1)
    want = [_moved(c, x, [path], [0]) for x in (c.k, c.v)]
    bt, lens, offs, cu = c.device()
    pkv.accept_tokens(c.pool, 0, bt, lens, offs, cu, table, count)
    assert torch.equal(c.k, want[0]) and torch.equal(c.v, want[1])


@pytest.mark.parametrize("validate", [False, True])
@pytest.mark.parametrize("path,count,error", [
    ([0, 2, 2], 3, "PKV_ERR_INDEX"), ([2, 1], 2, "PKV_ERR_INDEX"), ([0, 6], 2, "PKV_ERR_INDEX"),
    ([-1, 3], 2, "PKV_ERR_INDEX"), ([1, 2, 3], 4, "PKV_ERR_CAPACITY"), ([1, 2], -1, "PKV_ERR_CAPACITY"),
])
def test_accept_bad_paths(dev, path, count, error, validate):
    """A bad path moves nothing of its sequence; without validate mode the others move."""
    c, table, _ = _accept_case(dev, "bf16", 2, 64, 16, [40, 40], [6, 6], [[0, 3, 5], [0, 3, 5]])
    table = table[:, :3].contiguous()
    table[1, :len(path)] = _t(path, dev)
    good = [[0, 3, 5], []]
    want = [x.clone() if validate else _moved(c, x, good, range(3)) for x in (c.k, c.v)]
    bt, lens, offs, cu = c.device()
    pkv.set_validate(validate)
    try:
        if validate:
            with pytest.raises(PkvError) as e:
                pkv.accept_tokens(c.pool, -1, bt, lens, offs, cu, table, _t([3, count], dev))
            assert e.value.name == error
        else:
            pkv.accept_tokens(c.pool, -1, bt, lens, offs, cu, table, _t([3, count], dev))
            assert pkv.device_error() == error
    finally:
        pkv.set_validate(False)
    assert torch.equal(c.k, want[0]) and torch.equal(c.v, want[1])
    assert pkv.device_error() == "PKV_OK"


# ---- bad sequences and blocks -------------------------------------------------------

def _calls(c, mask):
    n = int(c.new.max())
    return {"window": lambda out: _window(c, 20, 3, out),
            "prefill": lambda out: _prefill(c, 20, 3, None, out),
            "tree": lambda out: _tree(c, mask, None, 0, 0, n, out)}


@pytest.mark.parametrize("what", ["window", "prefill", "tree"])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f32", 64)])
def test_bad_sequences(dev, what, dtype, D):
    """A sequence with bad numbers is skipped (windowed decode: gives zeros), one with a bad block
    id leaves it out; the others are computed as without them; validate mode names the error."""
    new = [1, 1, 1] if what == "window" else [20, 12, 20]

    def case():
        c = Case(dev, dtype, 2, 4, D, 16, [100, 60, 90], new, seed=21, offsets=False)
        trees = [np.tril(np.ones((n, n))) for n in new]
        return c, (_tree_args(c, trees, [np.zeros(n, np.int64) for n in new], 1)[0])

    c, mask = case()
    good = _calls(c, mask)[what](torch.full_like(c.q, 7.0))
    mid = slice(int(c.cu[1]), int(c.cu[2]))
    for field, value, error in (("lens", 1000, "PKV_ERR_CAPACITY"), ("lens", -1, "PKV_ERR_CAPACITY"),
                                ("offs", 16, "PKV_ERR_CAPACITY"), ("offs", -1, "PKV_ERR_CAPACITY"),
                                ("lens", 5, "PKV_ERR_CAPACITY"), ("table", 1 << 30, "PKV_ERR_INDEX"),
                                ("table", -1, "PKV_ERR_INDEX")):
        if field == "lens" and value == 5 and what == "window":
            continue
        c, mask = case()
        if field == "table":
            c.table[1, 3] = value
        else:
            getattr(c, field)[1] = value
        pkv.set_validate(True)
        try:
            out = torch.full_like(c.q, 7.0)
            with pytest.raises(PkvError) as e:
                _calls(c, mask)[what](out)
            assert e.value.name == error and bool((out == 7.0).all())
        finally:
            pkv.set_validate(False)
        got = _calls(c, mask)[what](torch.full_like(c.q, 7.0))
        assert pkv.device_error() == error
        keep = torch.ones(len(got), dtype=torch.bool, device=dev)
        keep[mid] = False
        # (the split of a tree's work follows the batch: the same to rounding)
        diff = (got[keep].float() - good[keep].float()).abs().max()
        assert float(diff) <= (2.0 ** -7 if dtype == "bf16" else 1e-5)
        if field != "table":
            assert bool((got[mid] == (0.0 if what == "window" else 7.0)).all())
        else:
            assert bool(got[mid].isfinite().all())


def test_bad_cu_q(dev):
    """Query ranges outside q, below zero or longer than the bound are not touched."""
    c = Case(dev, "bf16", 2, 4, 128, 16, [100, 60, 90], [20, 12, 20], seed=22)
    bt, lens, offs, _ = c.device()
    ws = _workspace(c, 20)
    for cu in ([0, 20, 32, 60], [0, 20, 90, 100], [-20, 0, 12, 32], [0, 20, 12, 32]):
        for what in ("prefill", "tree"):
            out = torch.full_like(c.q, 7.0)
            dcu = _t(cu, dev, torch.int64)
            if what == "prefill":
                pkv.prefill_attention_window(c.pool, c.layer, c.q, c.scale, bt, lens, offs, dcu, 20, 30, out)
            else:
                pkv.decode_attention_tree(c.pool, c.layer, c.q, c.scale, bt, lens, offs, dcu, 20, None, out, ws)
            assert pkv.device_error() == "PKV_ERR_CAPACITY"
            assert bool(out.isfinite().all())


def test_workspace_too_small(dev):
    c = Case(dev, "bf16", 2, 4, 128, 16, [100], [20])
    bt, lens, offs, cu = c.device()
    ws = _workspace(c, 20)
    out = torch.full_like(c.q, 7.0)
    for w, at in ((ws[:-1], 0), (ws[8:], 8)):
        with pytest.raises(PkvError) as e:
            pkv.decode_attention_tree(c.pool, c.layer, c.q, c.scale, bt, lens, offs, cu, 20, None, out, w)
        assert e.value.name == "PKV_ERR_WORKSPACE", at
    assert bool((out == 7.0).all())


# ---- together, as a server uses them --------------------------------------------------

@pytest.mark.parametrize("dtype,D,window", [("bf16", 128, 0), ("bf16", 128, 40), ("i8", 64, 0), ("f32", 64, 25)])
def test_a_verified_step(dev, dtype, D, window):
    """Drafted tokens stored with their tree positions, verified, the accepted path kept: the
    cache then holds what appending that path alone gives, and the path's outputs are those of a chain."""
    H, G, bs, ctx, n = 2, 4, 16, 75, 12
    io = torch.float32 if dtype == "f32" else torch.bfloat16
    path = [0, 3, 7, 8]

    def fresh():
        return Case(dev, dtype, H, G, D, bs, [ctx + n], [n], seed=31, layers=1, offsets=True)

    sees = np.zeros((n, n), bool)
    depth = np.zeros(n, np.int64)
    parent = [-1, -1, 0, 0, 1, 2, 3, 3, 7, 7, 8, 4]
    for i, a in enumerate(parent):
        if a >= 0:
            sees[i], depth[i] = sees[a], depth[a] + 1
        sees[i, i] = True
    a, b = fresh(), fresh()
    gen = torch.Generator(device=dev)
    gen.manual_seed(5)
    q, k, v = (torch.randn((n, h, D), generator=gen, device=dev).to(io) for h in (H * G, H, H))
    rope, zero = pkv.Rope(D), torch.zeros(n, dtype=torch.int32, device=dev)
    bt, lens, offs, cu = a.device()
    # the tree: rows in drafted order, angles by depth
    turned = torch.empty_like(q)
    order = _t(ctx + np.arange(n), dev)
    mask, pos = _tree_args(a, [sees], [depth], 1)
    pkv.rope_append(a.pool, 0, rope, bt, offs, zero, order, q, k, v, turned, rope_pos=pos)
    out = torch.empty_like(q)
    pkv.decode_attention_tree(a.pool, 0, turned, a.scale, bt, lens, offs, cu, n, mask, out,
                              _workspace(a, n), q_pos=pos, window=window, sink=2)
    pkv.accept_tokens(a.pool, -1, bt, lens, offs, cu, _t([path], dev), _t([len(path)], dev))
    # the path alone: a chain
    m = len(path)
    idx = torch.tensor(path, device=dev)
    cut = torch.empty((m, H * G, D), dtype=io, device=dev)
    short = _t([ctx + m], dev)
    pkv.rope_append(b.pool, 0, rope, bt, offs, zero[:m].contiguous(), order[:m].contiguous(), q[idx], k[idx],
                    v[idx], cut)
    chain = torch.empty_like(cut)
    scu = _t([0, m], dev, torch.int64)
    pkv.decode_attention_tree(b.pool, 0, cut, b.scale, bt, short, offs, scu, m, None, chain,
                              _workspace(b, m), window=window, sink=2)
    again = torch.empty_like(cut)
    if window:
        pkv.prefill_attention_window(b.pool, 0, cut, b.scale, bt, short, offs, scu, m, window, again, sink=2)
    else:
        pkv.prefill_attention_window(b.pool, 0, cut, b.scale, bt, short, offs, scu, m, 1 << 20, again)
    tol = 2.0 ** -6 if io is torch.bfloat16 else 2e-5
    assert torch.equal(turned[idx], cut)
    assert float((out[idx].float() - chain.float()).abs().max()) <= tol
    assert float((again.float() - chain.float()).abs().max()) <= tol
    if window == 0:
        # the last token of the path by the single-token call, over the moved rows
        one = torch.empty((1, H * G, D), dtype=io, device=dev)
        pkv.decode_attention_window(a.pool, 0, cut[-1:].contiguous(), a.scale, bt, short, offs, 1 << 20, one)
        assert float((one.float() - chain[-1:].float()).abs().max()) <= tol
    # the kept rows are those of the chain, to the bit (an int8 row's padding holds nothing)
    p = int(a.offs[0]) + ctx + np.arange(m)
    blk, row = torch.from_numpy(a.table[0, p // bs]).to(dev), torch.from_numpy(p % bs).to(dev)
    for x, y in ((a.k, b.k), (a.v, b.v)):
        held = H * D + 4 * H if dtype == "i8" else None
        assert torch.equal(x[blk, 0, row][..., :held], y[blk, 0, row][..., :held])
    assert pkv.device_error() == "PKV_OK"


def test_capture_streams_and_two_calls_at_once(dev):
    """Each call captured and replayed on another stream with new inputs in place, and two streams at once
    with a workspace each."""
    c = Case(dev, "bf16", 2, 4, 128, 16, [500, 80, 300], [16, 16, 16], seed=41)
    w = Case(dev, "bf16", 2, 4, 128, 16, [500, 80, 300], [1, 1, 1], seed=42)
    bt, lens, offs, cu = c.device()
    wbt, wlens, woffs, _ = w.device()
    outs = [torch.full_like(c.q, 7.0), torch.full_like(c.q, 7.0), torch.full_like(w.q, 7.0)]
    ws = _workspace(c, 16)
    path, count = _t([[0, 1, 2, 3]] * 3, dev), _t([4] * 3, dev)

    def step():
        pkv.prefill_attention_window(c.pool, c.layer, c.q, c.scale, bt, lens, offs, cu, 16, 50, outs[0], sink=2)
        pkv.decode_attention_tree(c.pool, c.layer, c.q, c.scale, bt, lens, offs, cu, 16, None, outs[1], ws)
        pkv.decode_attention_window(w.pool, w.layer, w.q, w.scale, wbt, wlens, woffs, 50, outs[2], sink=2)
        pkv.accept_tokens(c.pool, -1, bt, lens, offs, cu, path, count)

    step()
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        step()
    fresh = torch.randn_like(c.q.float()).to(c.q.dtype)
    c.q.copy_(fresh)
    step()
    want = [o.clone() for o in outs]
    for o in outs:
        o.fill_(7.0)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graph.replay()
    side.synchronize()
    for o, x in zip(outs, want):
        assert torch.equal(o, x)
    # two streams
    res, spaces = [torch.empty_like(c.q) for _ in range(2)], [_workspace(c, 16) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for o, x, s in zip(res, spaces, streams):
            with torch.cuda.stream(s):
                pkv.decode_attention_tree(c.pool, c.layer, c.q, c.scale, bt, lens, offs, cu, 16, None, o, x)
    torch.cuda.synchronize()
    assert torch.equal(res[0], want[1]) and torch.equal(res[1], want[1])
