"""GPU parity of sparse decode against the oracle in 64 bits: key bounds and
selections are whole numbers and have to be equal; attention is held to error
bounds.

Tolerance of the attention.  Let A be the weighted mean of |V| (the oracle
returns it), S the largest sum of |q| |k| over the keys, n the keys.
 * scores: a product of length D in fp32, any order, D + 8 roundings of
   2^-23 S scale (tensor cores may truncate), and exp2 of it, 2^-21: a weight
   is off by d = scale 2^-23 (D + 8) S + 2^-21 of itself, numerator and sum: 2 d A;
 * weights rounded for the product with V, half a step: bf16 in two parts,
   2^-16 A; int8 pools: fp16 2^-11 A, and weights (times V scales) below the smallest
   normal fp16 by 2^-25 of the largest V: n 2^-25 max|V|; fp32: none;
 * sums of n terms in fp32: n 2^-23 A;
 * the output's rounding, half a step of its value."""

from types import SimpleNamespace

import numpy as np
import pytest
import torch

from oracle import quant as Q
from oracle import rope as R
from oracle import sparse as SP
import oracle
import paged_kv_cache_blk_gb300 as pkv
from workloads import PoolSpec, fill_pool, fill_pool_i8, new_pool, rand_rows, small_workload
from workloads import to_numpy_bits

from gpu_util import dev_batch, gpu_decode, need_gpu, widen_out

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    d = need_gpu()
    pkv.set_validate(False)
    pkv.device_error(clear=True)
    return d


def _io(dtype):
    return "f32" if dtype == "f32" else "bf16"


def _make_pool(spec, layer, seed, dev):
    if spec.dtype == "i8":
        k = torch.zeros(spec.shape, dtype=torch.uint8, device=dev)
        v = torch.zeros_like(k)
        fill_pool_i8(k, v, spec, layer, seed)
        return pkv.Pool(k, v, spec.num_kv_heads, spec.head_dim)
    k, v = new_pool(spec, dev)
    fill_pool(k, v, spec, layer, seed)
    return pkv.Pool(k, v)


def _layer_values(t, spec, layer):
    """A layer of a cache as the library's fp32 values: [N, bs, H, D]."""
    if spec.dtype != "i8":
        return t[:, layer].float().cpu().numpy()
    rows = to_numpy_bits(t[:, layer].contiguous()).reshape(-1, spec.row_bytes)
    codes, scales = Q.unpack_rows(rows, spec.num_kv_heads, spec.head_dim)
    x = codes.astype(np.float32) * scales[..., None]
    return x.reshape(spec.num_blocks, spec.block_size, spec.num_kv_heads, spec.head_dim)


def _case(dev, dtype, H, D, bs, lens, seed, num_blocks=None, **kw):
    need = sum(-(-(n + bs) // bs) for n in lens) + kw.get("shared_prefix", 0) + 2
    w = small_workload(seed=seed, num_blocks=num_blocks or need, num_kv_heads=H, head_dim=D,
                       block_size=bs, lens=lens, dtype=_io(dtype), **kw)
    spec = PoolSpec(w.pool.num_blocks, w.pool.num_layers, bs, H, D, dtype)
    return w, spec, _make_pool(spec, w.layer, seed + 1, dev)


def _t(a, dev, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev, dtype)


# ---- key bounds -----------------------------------------------------------------

def _bounds_ref(w, spec, kvals, first=None):
    """{block: (codes [H, 2, D], exponents [H])} of the blocks an update names."""
    out, bs = {}, spec.block_size
    for b in range(w.batch.batch):
        n, off = int(w.batch.seq_lens[b]), int(w.batch.offsets[b])
        f = 0 if first is None else max(0, int(first[b]))
        if f >= n:
            continue
        for j in range((off + f) // bs, (off + n - 1) // bs + 1):
            blk = int(w.batch.block_tables[b, j])
            rows = kvals[blk][:min(bs, off + n - j * bs)]
            got = [SP.block_bounds(rows[:, g]) for g in range(spec.num_kv_heads)]
            out[blk] = (np.array([c for c, _ in got]), np.array([e for _, e in got]))
    return out


def _check_bounds(bounds, before, w, spec, kvals, first=None):
    ref = _bounds_ref(w, spec, kvals, first)
    codes, scales = bounds.codes.cpu().numpy(), bounds.scales.cpu().numpy()
    want_c, want_s = (x.copy() for x in before)
    for blk, (c, e) in ref.items():
        want_c[blk, w.layer] = c + 128
        want_s[blk, w.layer] = np.exp2(e.astype(np.float32))
    assert np.array_equal(codes, want_c) and np.array_equal(scales, want_s)
    return len(ref)


@pytest.mark.parametrize("dtype,H,D,bs,lens", [
    ("bf16", 8, 128, 16, [1, 16, 17, 0, 250]), ("bf16", 1, 64, 8, [70, 3]),
    ("bf16", 3, 64, 1, [5, 1]), ("bf16", 5, 128, 64, [64, 65, 200]),
    ("f32", 2, 128, 16, [33, 100]), ("f32", 7, 64, 32, [1, 90]),
    ("i8", 8, 128, 16, [40, 16, 1]), ("i8", 3, 64, 8, [77]), ("i8", 1, 128, 1024, [1100]),
])
def test_bounds(dev, dtype, H, D, bs, lens):
    w, spec, pool = _case(dev, dtype, H, D, bs, lens, 5)
    bounds = pkv.BlockBounds.for_pool(pool)
    bounds.codes.fill_(7)
    bounds.scales.fill_(-3.0)
    before = bounds.codes.cpu().numpy(), bounds.scales.cpu().numpy()
    bt, ln, offs, _ = dev_batch(w.batch, dev)
    kvals = _layer_values(pool.k_cache, spec, w.layer)
    pkv.update_block_bounds(pool, w.layer, bounds, bt, ln, offs)
    _check_bounds(bounds, before, w, spec, kvals)
    # the blocks of the last tokens only
    bounds.codes.fill_(9)
    bounds.scales.fill_(-1.0)
    before = bounds.codes.cpu().numpy(), bounds.scales.cpu().numpy()
    first = np.array([n - 1 if i % 2 else n - 20 for i, n in enumerate(lens)])
    pkv.update_block_bounds(pool, w.layer, bounds, bt, ln, offs, _t(first, dev))
    _check_bounds(bounds, before, w, spec, kvals, first)
    assert pkv.device_error() == "PKV_OK"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bounds_of_awkward_values(dev, dtype):
    """Zeros, subnormals, the type's extremes, infinities and NaN."""
    w, spec, pool = _case(dev, dtype, 1, 64, 4, [4] * 12, 15, offsets=False, num_layers=1, layer=0)
    top = float(torch.finfo(pool.dtype).max)
    tiny = float(torch.finfo(pool.dtype).tiny)
    k = torch.zeros_like(pool.k_cache)
    fills = [0.0, -0.0, tiny / 4, -tiny, top, -top, float("inf"), -float("inf"), float("nan"),
             127 * 2.0 ** -3, 127.5 * 2.0 ** -3, 2.0 ** -44]
    for b, x in enumerate(fills):
        blk = int(w.batch.block_tables[b, 0])
        k[blk] = torch.randn(k[blk].shape, device=dev).to(k.dtype) * (0 if b < 4 or b == 11 else 1)
        k[blk, 0, b % 4, 0, 3 * b] = x
    pool.k_cache.copy_(k)
    bounds = pkv.BlockBounds.for_pool(pool)
    bounds.codes.fill_(7)
    bounds.scales.fill_(-3.0)
    before = bounds.codes.cpu().numpy(), bounds.scales.cpu().numpy()
    bt, ln, offs, _ = dev_batch(w.batch, dev)
    pkv.update_block_bounds(pool, 0, bounds, bt, ln, offs)
    _check_bounds(bounds, before, w, spec, _layer_values(pool.k_cache, spec, 0))


def test_bounds_of_shared_blocks_and_errors(dev):
    """Sequences that share prefix blocks at different offsets write the same
    bytes; bad sequences and blocks are skipped and reported."""
    w, spec, pool = _case(dev, "bf16", 2, 128, 16, [60, 75, 90, 64], 25, shared_prefix=3)
    bounds = pkv.BlockBounds.for_pool(pool)
    bounds.codes.fill_(7)
    bounds.scales.fill_(-3.0)
    before = bounds.codes.cpu().numpy(), bounds.scales.cpu().numpy()
    bt, ln, offs, _ = dev_batch(w.batch, dev)
    kvals = _layer_values(pool.k_cache, spec, w.layer)
    for _ in range(3):
        pkv.update_block_bounds(pool, w.layer, bounds, bt, ln, offs)
        _check_bounds(bounds, before, w, spec, kvals)
    assert pkv.device_error() == "PKV_OK"
    bad = ln.clone()
    bad[1] = 10000
    args = (pool, w.layer, bounds, bt, bad, offs)
    pkv.update_block_bounds(*args)
    assert pkv.device_error() == "PKV_ERR_CAPACITY"
    tb = bt.clone()
    tb[0, 3] = spec.num_blocks
    pkv.update_block_bounds(pool, w.layer, bounds, tb, ln, offs)
    assert pkv.device_error() == "PKV_ERR_INDEX"
    _check_bounds(bounds, before, w, spec, kvals)
    pkv.set_validate(True)
    try:
        with pytest.raises(pkv.PkvError):
            pkv.update_block_bounds(*args)
    finally:
        pkv.set_validate(False)


# ---- selection --------------------------------------------------------------------

def _queries(rng, lens, q):
    """q queries a sequence at random positions, a tenth of the list padding."""
    seq = np.repeat(np.arange(len(lens)), q)
    pos = np.array([rng.integers(0, lens[b]) if lens[b] else 0 for b in seq])
    seq = np.where((rng.random(len(seq)) < 0.1) | (np.asarray(lens)[seq] == 0), -1, seq)
    return seq.astype(np.int32), pos.astype(np.int32)


def _random_bounds(pool, rng, dev, ties):
    """Bounds of no particular keys; with `ties`, of few different values."""
    shape = (pool.num_blocks, pool.num_layers, pool.num_kv_heads)
    if ties:
        pick = rng.integers(0, 3, size=shape)
        codes = np.array([140, 120, 130], np.uint8)[pick][..., None, None] \
            * np.ones((2, pool.head_dim), np.uint8)
        scales = np.exp2(rng.integers(0, 2, size=shape).astype(np.float32) - 3)
    else:
        codes = rng.integers(1, 256, size=shape + (2, pool.head_dim), dtype=np.uint8)
        codes = np.sort(codes, axis=3)[..., ::-1, :]
        scales = np.exp2(rng.integers(-6, -3, size=shape).astype(np.float32))
    return pkv.BlockBounds(_t(codes, dev, torch.uint8), _t(scales, dev, torch.float32))


def _select_ref(q, w, bounds, layer, seq, pos, H, bs, K, sink, recent):
    codes = bounds.codes.cpu().numpy().astype(np.int64) - 128
    scales = bounds.scales.cpu().numpy()
    T, G = q.shape[0], q.shape[1] // H
    sel = np.full((T, H, K), -1, np.int32)
    count = np.zeros((T, H), np.int32)
    for t in range(T):
        if seq[t] < 0:
            continue
        n = (int(w.batch.offsets[seq[t]]) + int(pos[t])) // bs + 1
        blk = w.batch.block_tables[seq[t], :n]
        for g in range(H):
            s = SP.block_scores(q[t, g * G:(g + 1) * G], codes[blk, layer, g], scales[blk, layer, g])
            best = SP.select(s, K, sink, recent)
            sel[t, g, :len(best)], count[t, g] = best, len(best)
    return sel, count


def _run_select(dev, dtype, H, G, D, bs, lens, K, sink, recent, q_per=2, ties=False, seed=7,
                scale_q=1.0):
    w, spec, pool = _case(dev, dtype, H, D, bs, lens, seed)
    rng = np.random.default_rng(seed + 3)
    seq, pos = _queries(rng, lens, q_per)
    bounds = _random_bounds(pool, rng, dev, ties)
    q = rand_rows((len(seq), H * G, D), _io(dtype), seed + 4, dev) * scale_q
    sel = torch.full((len(seq), H, K), 77, dtype=torch.int32, device=dev)
    cnt = torch.full((len(seq), H), 77, dtype=torch.int32, device=dev)
    bt, _, offs, _ = dev_batch(w.batch, dev)
    pkv.select_blocks(pool, w.layer, bounds, q, bt, offs, _t(seq, dev), _t(pos, dev), sel, cnt,
                      sink=sink, recent=recent)
    want_s, want_c = _select_ref(widen_out(q), w, bounds, w.layer, seq, pos, H, bs, K, sink, recent)
    assert np.array_equal(cnt.cpu().numpy(), want_c)
    assert np.array_equal(sel.cpu().numpy(), want_s)
    assert pkv.device_error() == "PKV_OK"


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("dtype,H,G,D,bs,lens,K,sink,recent", [
    ("bf16", 8, 4, 128, 16, [1000, 1, 17, 0, 400], 16, 1, 2),
    ("bf16", 2, 1, 64, 8, [3000, 700], 33, 0, 0), ("bf16", 1, 16, 128, 16, [2000, 900], 20, 4, 4),
    ("f32", 4, 3, 128, 16, [900, 64], 10, 0, 1), ("f32", 1, 9, 64, 1, [300, 40], 7, 2, 5),
    ("i8", 3, 5, 128, 32, [2500], 11, 1, 1), ("bf16", 2, 8, 64, 1024, [9000], 3, 1, 1),
    ("f32", 2, 16, 128, 8, [600], 1, 0, 0), ("bf16", 4, 2, 128, 16, [5000], 300, 0, 0),
])
def test_select(dev, dtype, H, G, D, bs, lens, K, sink, recent, ties):
    _run_select(dev, dtype, H, G, D, bs, lens, K, sink, recent, ties=ties)


@pytest.mark.parametrize("n,K", [(130000, 200), (70000, 5000), (40000, 39999)])
def test_select_long(dev, n, K):
    """Many entries a query: clusters of several CTAs."""
    _run_select(dev, "bf16", 1, 2, 64, 1, [n], K, 3, 2, q_per=1, seed=17)


@pytest.mark.parametrize("n", [7000, 9500, 11500, 14000])
def test_select_rows_of_one_cta(dev, n):
    """Many rows of long tables: one CTA holds all scores of a row, up to and
    past 48 KB of them."""
    _run_select(dev, "bf16", 8, 1, 64, 1, [n, 700], 40, 1, 1, q_per=21, seed=67)


def test_select_many_queries(dev):
    """More rows than CTAs are resident, one CTA a row."""
    _run_select(dev, "bf16", 8, 2, 64, 16, [300, 900, 77], 9, 1, 1, q_per=30, seed=27)


@pytest.mark.parametrize("G,D", [(2, 64), (12, 128)])
@pytest.mark.parametrize("q_per", [2, 4, 9, 13, 24])
def test_select_many_rows(dev, G, D, q_per):
    """Rows for a part of the SMs up to several for each; clusters of every size."""
    _run_select(dev, "bf16", 8, G, D, 4, [6300, 900], 12, 1, 1, q_per=q_per, seed=77)


@pytest.mark.parametrize("scale_q", [0.0, 1e-30, 1e30])
def test_select_query_range(dev, scale_q):
    _run_select(dev, "f32", 2, 2, 64, 16, [800], 5, 0, 1, scale_q=scale_q, seed=37)


def test_select_forced_only_and_bad_input(dev):
    _run_select(dev, "bf16", 2, 2, 64, 16, [800, 90], 7, 3, 4, seed=47)
    w, spec, pool = _case(dev, "bf16", 2, 64, 16, [400, 300], 57)
    rng = np.random.default_rng(58)
    bounds = _random_bounds(pool, rng, dev, False)
    bt, _, offs, _ = dev_batch(w.batch, dev)
    cap = bt.shape[1] * 16
    q = rand_rows((5, 4, 64), "bf16", 59, dev)
    sel = torch.full((5, 2, 4), 77, dtype=torch.int32, device=dev)
    cnt = torch.full((5, 2), 77, dtype=torch.int32, device=dev)
    seq, pos = _t([2, 0, -1, 1, -5], dev), _t([0, cap, 5, -1, 5], dev)
    pkv.select_blocks(pool, w.layer, bounds, q, bt, offs, seq, pos, sel, cnt)
    assert pkv.device_error() in ("PKV_ERR_INDEX", "PKV_ERR_CAPACITY")
    assert not cnt.any() and bool((sel == -1).all())
    # an entry with an invalid block id is not read and scores lowest
    tb = bt.clone()
    tb[0, 5] = spec.num_blocks + 3
    pkv.select_blocks(pool, w.layer, bounds, q[:1], tb, offs, _t([0], dev), _t([399], dev), sel[:1],
                      cnt[:1])
    assert pkv.device_error() == "PKV_ERR_INDEX"
    assert not bool((sel[:1] == 5).any()) and bool((cnt[:1] == 4).all())


# ---- attention -----------------------------------------------------------------------

def _entries(rng, seq, pos, w, H, K, bs, full=False):
    """Lists of table entries in random order with holes and entries past the query."""
    sel = np.full((len(seq), H, K), -1, np.int32)
    for t in range(len(seq)):
        if seq[t] < 0:
            continue
        n = (int(w.batch.offsets[seq[t]]) + int(pos[t])) // bs + 1
        for g in range(H):
            x = rng.permutation(n)[:K]
            sel[t, g, :len(x)] = x
            if not full:
                sel[t, g, rng.random(K) < 0.2] = -1
                if rng.random() < 0.3:
                    sel[t, g, rng.integers(K)] = w.batch.block_tables.shape[1] - 1
                rng.shuffle(sel[t, g])
    return sel


def _check_attention(got, q, kvals, vvals, w, spec, seq, pos, sel, scale, untouched):
    H, D, bs = spec.num_kv_heads, spec.head_dim, spec.block_size
    G = q.shape[1] // H
    worst = 0.0
    for t in range(len(seq)):
        if seq[t] < 0:
            assert np.array_equal(got[t], untouched[t])
            continue
        table, off = w.batch.block_tables[seq[t]], int(w.batch.offsets[seq[t]])
        for g in range(H):
            x = q[t, g * G:(g + 1) * G]
            ref, mean, top = SP.sparse_attention(x, kvals[table, :, g], vvals[table, :, g],
                                                 sel[t, g], bs, off, int(pos[t]), scale)
            n = int((sel[t, g] >= 0).sum()) * bs
            d = abs(scale) * 2.0 ** -23 * (D + 8) * top[:, None] + 2.0 ** -21
            tol = (2 * d + n * 2.0 ** -23) * mean
            if spec.dtype == "f32":
                tol = tol + 2.0 ** -24 * np.abs(ref)
            elif spec.dtype == "bf16":
                tol = tol + 2.0 ** -16 * mean + 2.0 ** -8 * np.abs(ref) * 1.01
            else:
                vmax = np.abs(vvals[table, :, g]).max()
                tol = tol + 2.0 ** -11 * mean + n * 2.0 ** -25 * vmax + 2.0 ** -8 * np.abs(ref) * 1.01
            err = np.abs(got[t, g * G:(g + 1) * G] - ref)
            assert np.all(err <= tol + 1e-30), (t, g, float((err - tol).max()))
            worst = max(worst, float(err.max()))
    return worst


def _run_sparse(dev, dtype, H, G, D, bs, lens, K, q_per=2, seed=9, full=False, poison=True):
    w, spec, pool = _case(dev, dtype, H, D, bs, lens, seed)
    rng = np.random.default_rng(seed + 3)
    seq, pos = _queries(rng, lens, q_per)
    sel = _entries(rng, seq, pos, w, H, K, bs, full)
    kvals = _layer_values(pool.k_cache, spec, w.layer)
    vvals = _layer_values(pool.v_cache, spec, w.layer)
    if poison and dtype != "i8":
        # rows that no query sees hold NaN: other layers, rows outside the sequences
        seen = torch.zeros(pool.k_cache.shape[:3], dtype=torch.bool, device=dev)
        for t in range(len(seq)):
            if seq[t] >= 0:
                p = int(w.batch.offsets[seq[t]]) + np.arange(pos[t] + 1)
                seen[_t(w.batch.block_tables[seq[t]][p // bs], dev).long(), w.layer,
                     _t(p % bs, dev).long()] = True
        for c in (pool.k_cache, pool.v_cache):
            c.masked_fill_(~seen[..., None, None], float("nan"))
    q = rand_rows((len(seq), H * G, D), _io(dtype), seed + 4, dev)
    out = torch.full_like(q, 7.0)
    before = widen_out(out)
    bt, _, offs, _ = dev_batch(w.batch, dev)
    scale = D ** -0.5
    pkv.decode_attention_sparse(pool, w.layer, q, scale, bt, offs, _t(seq, dev), _t(pos, dev),
                                _t(sel, dev), out)
    _check_attention(widen_out(out), widen_out(q), kvals, vvals, w, spec, seq, pos, sel, scale,
                     before)
    assert pkv.device_error() == "PKV_OK"


@pytest.mark.parametrize("dtype,H,G,D,bs,lens,K", [
    ("bf16", 8, 4, 128, 16, [300, 1, 16, 17, 0], 9), ("bf16", 2, 1, 64, 8, [200, 3], 20),
    ("bf16", 1, 16, 128, 16, [500], 31), ("bf16", 3, 9, 64, 1, [40, 9], 25),
    ("bf16", 2, 3, 128, 64, [700, 64], 5), ("bf16", 1, 8, 64, 1024, [2100], 3),
    ("f32", 4, 3, 64, 32, [300, 1, 90], 6), ("f32", 2, 1, 128, 16, [260], 12),
    ("f32", 1, 16, 128, 8, [100, 50], 9), ("f32", 2, 7, 64, 2, [60], 22),
    ("f32", 3, 5, 128, 16, [70], 4), ("f32", 1, 12, 64, 16, [80], 5),
    ("i8", 8, 4, 128, 16, [300, 1, 17], 9), ("i8", 2, 16, 64, 8, [120], 11),
    ("i8", 3, 1, 64, 16, [99, 33], 5), ("i8", 1, 10, 128, 32, [400], 8), ("i8", 5, 2, 128, 1, [30], 13),
])
def test_sparse_attention(dev, dtype, H, G, D, bs, lens, K):
    _run_sparse(dev, dtype, H, G, D, bs, lens, K)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "i8"])
@pytest.mark.parametrize("D", [64, 128])
def test_sparse_attention_long_lists(dev, dtype, D):
    """More tiles than one lookup of a warp holds, on clusters of CTAs."""
    _run_sparse(dev, dtype, 1, 2, D, 16, [40000], 2300, q_per=1, seed=19, full=True)
    _run_sparse(dev, dtype, 2, 4, D, 16, [3000, 1500], 150, q_per=20, seed=29)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "i8"])
@pytest.mark.parametrize("H,G,D,bs,lens,K,q_per", [
    (8, 2, 64, 16, [300, 90, 20], 5, 15), (8, 1, 128, 8, [260, 200], 30, 23),
    (8, 4, 128, 16, [700], 40, 5), (4, 9, 64, 32, [500, 40], 12, 11),
    (1, 3, 128, 4, [900], 200, 2), (4, 5, 128, 2, [100, 60, 7], 40, 9),
])
def test_sparse_attention_many_rows(dev, dtype, H, G, D, bs, lens, K, q_per):
    """Rows for part of the SMs, for one CTA each and for several rounds; tiles of small blocks."""
    _run_sparse(dev, dtype, H, G, D, bs, lens, K, q_per=q_per, seed=71)


def test_sparse_equals_dense_on_every_entry(dev):
    """With all entries listed, pkv_decode_attention's result within both calls' bounds."""
    w, spec, pool = _case(dev, "bf16", 8, 128, 16, [900, 37, 512], 39)
    bt, ln, offs, _ = dev_batch(w.batch, dev)
    q = rand_rows((3, 32, 128), "bf16", 40, dev)
    dense = gpu_decode(pool, w.layer, q, 128 ** -0.5, w.batch, dev)
    K = bt.shape[1]
    sel = torch.arange(K, dtype=torch.int32, device=dev).expand(3, 8, K).contiguous()
    out = torch.empty_like(q)
    pkv.decode_attention_sparse(pool, w.layer, q, 128 ** -0.5, bt, offs,
                                torch.arange(3, dtype=torch.int32, device=dev), ln - 1, sel, out)
    assert (out.double() - dense.double()).abs().max().item() <= 2e-2


def test_offsets_past_32_bits(dev):
    """Blocks beyond 4 GiB of a cache."""
    H, D, bs, N = 8, 128, 64, 36000          # 131072 bytes a block and tensor: 4.7 GB
    k = torch.empty((N, 1, bs, H, D), dtype=torch.bfloat16, device=dev)
    v = torch.empty_like(k)
    pool = pkv.Pool(k, v)
    blocks = [N - 1, 3, N - 2, 33000, 0, N - 700]
    w = SimpleNamespace(layer=0, batch=SimpleNamespace(
        block_tables=np.array([blocks], np.int32), seq_lens=np.array([bs * 6 - 5]),
        offsets=np.array([2]), batch=1))
    for i, b in enumerate(blocks):
        k[b], v[b] = (rand_rows((1, bs, H, D), "bf16", 100 + 2 * i + j, dev) for j in (0, 1))
    spec = PoolSpec(N, 1, bs, H, D, "bf16")
    kv = {b: k[b, 0].float().cpu().numpy() for b in blocks}
    vv = {b: v[b, 0].float().cpu().numpy() for b in blocks}
    bt = _t(w.batch.block_tables, dev)
    one = lambda a: torch.tensor([a], dtype=torch.int32, device=dev)
    n, off = int(w.batch.seq_lens[0]), one(2)
    bounds = pkv.BlockBounds.for_pool(pool)
    pkv.update_block_bounds(pool, 0, bounds, bt, one(n), off)
    for blk, (c, e) in _bounds_ref(w, spec, kv).items():
        assert np.array_equal(bounds.codes[blk, 0].cpu().numpy().astype(int) - 128, c)
        assert np.array_equal(bounds.scales[blk, 0].cpu().numpy(), np.exp2(e))
    q = rand_rows((1, 16, D), "bf16", 140, dev)
    sel = torch.empty((1, H, 4), dtype=torch.int32, device=dev)
    cnt = torch.empty((1, H), dtype=torch.int32, device=dev)
    out = torch.empty_like(q)
    pkv.select_blocks(pool, 0, bounds, q, bt, off, one(0), one(n - 1), sel, cnt)
    pkv.decode_attention_sparse(pool, 0, q, 0.1, bt, off, one(0), one(n - 1), sel, out)
    new_k, new_v = rand_rows((1, H, D), "bf16", 141, dev), rand_rows((1, H, D), "bf16", 142, dev)
    assert pkv.device_error() == "PKV_OK"
    x, s = widen_out(q), sel.cpu().numpy()
    for g in range(H):
        K, V = (np.stack([c[b][:, g] for b in blocks]) for c in (kv, vv))
        ref, mean, top = SP.sparse_attention(x[0, 2 * g:2 * g + 2], K, V, s[0, g], bs, 2, n - 1, 0.1)
        tol = (2 * (0.1 * 2.0 ** -23 * (D + 8) * top[:, None] + 2.0 ** -21) + 256 * 2.0 ** -23
               + 2.0 ** -16) * mean + 2.0 ** -8 * np.abs(ref) * 1.01
        assert np.all(np.abs(widen_out(out)[0, 2 * g:2 * g + 2] - ref) <= tol)
    # and a store at the far end, at rotary position 0
    pkv.rope_append(pool, 0, pkv.Rope(D), bt, off, one(0), one(3), None, new_k, new_v, None,
                    rope_pos=one(0))
    assert torch.equal(k[N - 1, 0, 5], new_k[0]) and torch.equal(v[N - 1, 0, 5], new_v[0])


def test_sparse_special_lists(dev):
    """An entry twice counts twice; nothing listed, no keys seen or only
    scores of -inf give zeros; a NaN that is seen shows; bad input."""
    w, spec, pool = _case(dev, "f32", 2, 64, 16, [200, 120], 49, offsets=False)
    bt, _, offs, _ = dev_batch(w.batch, dev)
    q = rand_rows((2, 4, 64), "f32", 50, dev)
    seq, pos = _t([0, 1], dev), _t([199, 119], dev)

    def run(sel, seq=seq, pos=pos, bt=bt):
        out = torch.full_like(q, 7.0)
        s = torch.tensor(sel, dtype=torch.int32, device=dev).expand(2, 2, len(sel)).contiguous()
        pkv.decode_attention_sparse(pool, w.layer, q, 0.125, bt, offs, seq, pos, s, out)
        return out

    kv, vv = (_layer_values(c, spec, w.layer) for c in (pool.k_cache, pool.v_cache))
    twice = run([2, 5, 2])
    _check_attention(widen_out(twice), widen_out(q), kv, vv, w, spec, [0, 1], [199, 119],
                     np.broadcast_to([2, 5, 2], (2, 2, 3)), 0.125, None)
    assert not run([-1, -1, -9]).any() and not run([]).any()
    assert not run([3], pos=_t([10, 10], dev)).any()         # wholly past the query
    assert pkv.device_error() == "PKV_OK"
    run([bt.shape[1]])
    assert pkv.device_error() == "PKV_ERR_INDEX"
    tb = bt.clone()
    tb[:, 4] = spec.num_blocks
    tb[1, 4] = -1
    assert torch.equal(run([1, 4, 3], bt=tb), run([1, 3, -1]))
    assert pkv.device_error() == "PKV_ERR_INDEX"
    bad = run([0], seq=_t([7, 0], dev), pos=_t([0, 1 << 20], dev))
    assert not bad.any() and pkv.device_error() in ("PKV_ERR_INDEX", "PKV_ERR_CAPACITY")
    pad = run([0], seq=_t([-1, 1], dev))
    assert bool((pad[0] == 7).all()) and not bool((pad[1] == 7).any())
    blk = int(w.batch.block_tables[0, 2])
    pool.v_cache[blk, w.layer, 3, 1, 5] = float("nan")
    got = run([2, 5])
    assert bool(got[0, 2:, 5].isnan().all()) and int(got.isnan().sum()) == 2
    pool.v_cache[blk, w.layer, 3, 1, 5] = 0.0
    pool.k_cache[blk, w.layer] = -float("inf")
    q.abs_()
    assert not run([2])[0].any()
    assert torch.equal(run([2, 5])[0], run([5, -1])[0])
    pool.k_cache[blk, w.layer] = float("nan")
    assert bool(run([2, 5])[0].isnan().all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("top", [False, True])
def test_sparse_infinite_values(dev, dtype, top):
    """An infinite value that is seen is what the sum over its element becomes, whether its
    weight is a power of two (the row of the largest score) or not; other elements stay."""
    w, spec, pool = _case(dev, dtype, 2, 128, 16, [100], 61, offsets=False)
    bt, _, offs, _ = dev_batch(w.batch, dev)
    q = rand_rows((1, 8, 128), dtype, 62, dev)
    one = lambda a: torch.tensor([a], dtype=torch.int32, device=dev)
    sel = torch.tensor([[[0, 2, 3]] * 2], dtype=torch.int32, device=dev)
    out = torch.empty_like(q)

    def run():
        pkv.decode_attention_sparse(pool, w.layer, q, 128 ** -0.5, bt, offs, one(0), one(99), sel, out)
        return out.clone()

    clean = run()
    blk = int(w.batch.block_tables[0, 2])
    if top:
        # every head's largest score: 2 |q|^2 / sqrt(D) of one head, the others' below it
        q[:] = q[:, :1]
        pool.k_cache[blk, w.layer, 5] = 2 * q[0, 0]
        clean = run()
    pool.v_cache[blk, w.layer, 5, 0, 7] = float("inf")
    pool.v_cache[blk, w.layer, 5, 0, 70] = -float("inf")
    pool.v_cache[blk, w.layer, 5, 1, 126] = float("inf")
    got = run()
    want = clean.clone()
    want[0, :4, 7], want[0, :4, 70], want[0, 4:, 126] = float("inf"), -float("inf"), float("inf")
    assert torch.equal(got, want)


def test_sparse_nan_keys_and_infinite_scores(dev):
    w, spec, pool = _case(dev, "bf16", 1, 128, 16, [64], 59, offsets=False)
    bt, _, offs, _ = dev_batch(w.batch, dev)
    q = rand_rows((1, 4, 128), "bf16", 60, dev).abs()
    one = lambda a: torch.tensor([a], dtype=torch.int32, device=dev)

    def run(sel):
        out = torch.full_like(q, 7.0)
        pkv.decode_attention_sparse(pool, w.layer, q, 0.1, bt, offs, one(0), one(63),
                                    torch.tensor([[sel]], dtype=torch.int32, device=dev), out)
        return out

    blk = int(w.batch.block_tables[0, 1])
    pool.k_cache[blk, w.layer] = -float("inf")
    assert not run([1, -1]).any()
    assert torch.equal(run([1, 2]), run([-1, 2]))
    pool.k_cache[blk, w.layer, 0] = float("nan")
    assert bool(run([1, 2]).isnan().all())


# ---- together ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32", "i8"])
def test_a_server_with_sparse_decode(dev, dtype):
    """Prompts, then decode steps: allocator, rotary append, bounds, selection
    and attention, each step checked against the oracle on the pool's contents."""
    H, G, D, bs, K, N = 2, 4, 64, 8, 6, 96
    spec = PoolSpec(N, 2, bs, H, D, dtype)
    layer = 1
    pool = _make_pool(spec, layer, 71, dev)
    bounds = pkv.BlockBounds.for_pool(pool)
    rope = pkv.Rope(D, base=10000.0)
    freq = R.inv_freq(D, 10000.0)
    rng = np.random.default_rng(72)
    al = pkv.Allocator(N, bs)
    ids = list(range(4))
    MB = 32
    w = SimpleNamespace()

    def step(counts):
        old = [al.seq_info(i)[0] for i in ids]
        al.seq_append_batch(ids, counts)
        tables, ln, offs = al.seq_tables(ids, MB)
        w.batch = SimpleNamespace(block_tables=tables, seq_lens=ln, offsets=offs, batch=len(ln))
        seq = np.repeat(ids, counts).astype(np.int32)
        pos = np.concatenate([old[b] + np.arange(counts[b]) for b in ids]).astype(np.int32)
        T = len(seq)
        qkv = rand_rows((T, (G + 2) * H, D), _io(dtype), int(rng.integers(1 << 30)), dev)
        q, k, v = qkv[:, :G * H], qkv[:, G * H:G * H + H], qkv[:, G * H + H:]
        qr = torch.empty((T, G * H, D), dtype=qkv.dtype, device=dev)
        bt, dl, do = _t(tables, dev), _t(ln, dev), _t(offs, dev)
        ds, dp = _t(seq, dev), _t(pos, dev)
        pkv.rope_append(pool, layer, rope, bt, do, ds, dp, q, k, v, qr)
        pkv.update_block_bounds(pool, layer, bounds, bt, dl, do, _t(old, dev))
        sel = torch.empty((T, H, K), dtype=torch.int32, device=dev)
        cnt = torch.empty((T, H), dtype=torch.int32, device=dev)
        out = torch.empty_like(qr)
        pkv.select_blocks(pool, layer, bounds, qr, bt, do, ds, dp, sel, cnt, sink=1, recent=1)
        pkv.decode_attention_sparse(pool, layer, qr, D ** -0.5, bt, do, ds, dp, sel, out)
        assert pkv.device_error() == "PKV_OK"
        # q as the oracle turns it, K and V as they are stored now
        ref = R.rotate(widen_out(q), pos, freq, False)
        assert np.max(np.abs(widen_out(qr) - ref)) <= 2.0 ** (-8 if dtype != "f32" else -20) \
            * np.abs(ref).max()
        kv, vv = (_layer_values(c, spec, layer) for c in (pool.k_cache, pool.v_cache))
        live = _bounds_ref(w, spec, kv)
        codes = bounds.codes.cpu().numpy().astype(int) - 128
        for blk, (c, e) in live.items():
            assert np.array_equal(codes[blk, layer], c), blk
            assert np.array_equal(bounds.scales.cpu().numpy()[blk, layer], np.exp2(e))
        want, wc = _select_ref(widen_out(qr), w, bounds, layer, seq, pos, H, bs, K, 1, 1)
        assert np.array_equal(sel.cpu().numpy(), want) and np.array_equal(cnt.cpu().numpy(), wc)
        _check_attention(widen_out(out), widen_out(qr), kv, vv, w, spec, seq, pos, want, D ** -0.5,
                         None)

    for i in ids:
        al.seq_new(i, 0)
    for counts in ([37, 150, 1, 64], [1, 1, 1, 1], [1, 1, 1, 1], [3, 1, 2, 5], [1, 1, 1, 1]):
        step(counts)
    al.close()


def test_graph_replay_and_another_stream(dev):
    """The three calls captured together and replayed on new inputs, next to
    eager ones on another stream."""
    H, G, D, bs, K = 4, 4, 128, 16, 8
    w, spec, pool = _case(dev, "bf16", H, D, bs, [900, 333, 700], 81)
    bt, ln, offs, _ = dev_batch(w.batch, dev)
    seq = torch.arange(3, dtype=torch.int32, device=dev)
    pos = (ln - 1).to(torch.int32)
    q = rand_rows((3, H * G, D), "bf16", 82, dev)
    sides = []
    for _ in range(2):
        sides.append((pkv.BlockBounds.for_pool(pool),
                      torch.zeros((3, H, K), dtype=torch.int32, device=dev),
                      torch.zeros((3, H), dtype=torch.int32, device=dev), torch.zeros_like(q)))

    def call(side):
        b, sel, cnt, out = side
        pkv.update_block_bounds(pool, w.layer, b, bt, ln, offs)
        pkv.select_blocks(pool, w.layer, b, q, bt, offs, seq, pos, sel, cnt, sink=1, recent=1)
        pkv.decode_attention_sparse(pool, w.layer, q, D ** -0.5, bt, offs, seq, pos, sel, out)

    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        call(sides[0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(sides[0])
    for i in range(3):
        q.copy_(rand_rows(q.shape, "bf16", 90 + i, dev))
        pos.sub_(37)
        pool.k_cache.add_(0.01)
        torch.cuda.synchronize()
        g.replay()
        with torch.cuda.stream(other):
            call(sides[1])
        torch.cuda.synchronize()
        for a, b in zip(sides[0][1:], sides[1][1:]):
            assert torch.equal(a, b)
    assert pkv.device_error() == "PKV_OK"


def test_binding_refusals(dev):
    w, spec, pool = _case(dev, "bf16", 2, 64, 16, [100], 91)
    bt, ln, offs, _ = dev_batch(w.batch, dev)
    bounds = pkv.BlockBounds.for_pool(pool)
    q = rand_rows((1, 4, 64), "bf16", 92, dev)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)
    ok = dict(q=q, bt=bt, offs=offs, seq=i32(1), pos=i32(1), sel=i32(1, 2, 4))

    def select(cnt=None, bounds=bounds, **kw):
        a = {**ok, **kw}
        pkv.select_blocks(pool, 0, bounds, *a.values(), i32(1, 2) if cnt is None else cnt)

    def sparse(out=None, **kw):
        a = {**ok, **kw}
        pkv.decode_attention_sparse(pool, 0, a["q"], 0.1, a["bt"], a["offs"], a["seq"], a["pos"],
                                    a["sel"], torch.empty_like(q) if out is None else out)

    pkv.update_block_bounds(pool, 0, bounds, bt, ln, offs)
    select()
    sparse()
    for kw in (dict(q=q.float()), dict(q=q[..., :32]), dict(seq=i32(1).long()), dict(pos=i32(2)),
               dict(sel=i32(1, 1, 4)), dict(sel=i32(2, 2, 4)), dict(sel=i32(1, 2, 4).float()),
               dict(offs=i32(2)), dict(bt=bt.cpu()), dict(sel=i32(1, 2, 8)[..., ::2])):
        for f in (select, sparse):
            with pytest.raises(ValueError):
                f(**kw)
    with pytest.raises(ValueError):
        select(cnt=i32(1, 3))
    with pytest.raises(ValueError):
        sparse(out=q[..., :32])
    small = pkv.BlockBounds(bounds.codes[:1].contiguous(), bounds.scales[:1].contiguous())
    with pytest.raises(ValueError):
        select(bounds=small)
    with pytest.raises(ValueError):
        pkv.update_block_bounds(pool, 0, small, bt, ln, offs)
    with pytest.raises(ValueError):
        pkv.update_block_bounds(pool, 0, bounds, bt, ln[:0], offs)
    with pytest.raises(ValueError):
        pkv.BlockBounds(bounds.codes.float(), bounds.scales)
