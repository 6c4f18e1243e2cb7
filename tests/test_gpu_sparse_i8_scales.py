"""Sparse attention from int8 pools whose V scales differ widely, and rows of
int8 pools that no query sees.

Tolerance.  As in test_gpu_sparse: with A the weighted mean of |V| (element by
element), S the largest sum of |q| |k|, n the keys and d = scale 2^-23 (D + 8) S +
2^-21, scores and their exp2 cost 2 d A and the fp32 sums n 2^-23 A.  The products of
weights and V scales enter the product with V as an fp16 and the fp16 of what it
leaves, each rounding at most half a step of 2^-11: 2^-22 A, or, below the normal numbers
of fp16, 2^-25 of a unit in which the largest product P is at least 2^2: 2^-27 P, times a
code of at most 127, for each key.  A weight below the smallest normal fp32 counts as
zero, which loses n 2^-126 of the largest V that is seen, and so does a product of one and
a scale, which meets a code of at most 127: n 2^-119.  The output is bf16: 2^-8 of its
value."""

import numpy as np
import pytest
import torch

from oracle import quant as Q
from oracle import sparse as SP
import paged_kv_cache_blk_gb300 as pkv
from workloads import rand_rows, to_numpy_bits

from gpu_util import dev_batch, need_gpu, widen_out
from test_gpu_sparse import _case, _entries, _queries, _t

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    d = need_gpu()
    pkv.set_validate(False)
    pkv.device_error(clear=True)
    return d


def _scales(cache, spec):
    """The scales of an int8 cache as a writable fp32 view [N, L, bs, H]."""
    hd = spec.num_kv_heads * spec.head_dim
    return cache[..., hd:hd + 4 * spec.num_kv_heads].view(torch.float32)


def _values(cache, spec, layer):
    """A layer of an int8 cache in 64 bits: [N, bs, H, D]."""
    rows = to_numpy_bits(cache[:, layer].contiguous()).reshape(-1, spec.row_bytes)
    codes, scales = Q.unpack_rows(rows, spec.num_kv_heads, spec.head_dim)
    with np.errstate(invalid="ignore"):
        x = codes.astype(np.float64) * scales.astype(np.float64)[..., None]
    return x.reshape(spec.num_blocks, spec.block_size, spec.num_kv_heads, spec.head_dim)


def _check(out, q, pool, w, spec, seq, pos, sel, scale):
    kv, vv = (_values(c, spec, w.layer) for c in (pool.k_cache, pool.v_cache))
    vs = _scales(pool.v_cache, spec)[:, w.layer].double().cpu().numpy()
    H, D, bs = spec.num_kv_heads, spec.head_dim, spec.block_size
    G = q.shape[1] // H
    got, x = widen_out(out).astype(np.float64), widen_out(q)
    for t in range(len(seq)):
        if seq[t] < 0:
            continue
        table, off = w.batch.block_tables[seq[t]], int(w.batch.offsets[seq[t]])
        for g in range(H):
            rows = slice(g * G, (g + 1) * G)
            ref, mean, top = SP.sparse_attention(x[t, rows], kv[table, :, g], vv[table, :, g], sel[t, g],
                                                 bs, off, int(pos[t]), scale)
            at = [j * bs + r for j in sel[t, g] if j >= 0 for r in range(bs)
                  if off <= j * bs + r <= off + int(pos[t])]
            n = len(at)
            if n == 0:
                assert not got[t, rows].any()
                continue
            at = (table[np.array(at) // bs], np.array(at) % bs, g)
            vmax = np.abs(vv[at]).max()
            s = x[t, rows].astype(np.float64) @ kv[at].T * scale
            wt = np.exp(s - s.max(-1, keepdims=True))
            wt /= wt.sum(-1, keepdims=True)
            most = (wt * np.abs(vs[at])).max(-1)[:, None]
            d = abs(scale) * 2.0 ** -23 * (D + 8) * top[:, None] + 2.0 ** -21
            tol = (2 * d + n * 2.0 ** -23 + 2.0 ** -22) * mean + 2.0 ** -8 * np.abs(ref) * 1.01 \
                + n * (127 * 2.0 ** -27 * most + 2.0 ** -126 * vmax + 2.0 ** -119)
            err = np.abs(got[t, rows] - ref)
            assert np.all(err <= tol), (t, g, float(np.nanmax(err)), float(np.abs(ref).max()))


@pytest.mark.parametrize("D,H,G,bs", [(128, 2, 4, 16), (64, 1, 2, 16), (128, 1, 16, 8), (64, 3, 5, 64)])
@pytest.mark.parametrize("where", ["first", "middle", "last"])
@pytest.mark.parametrize("bits", [12, 20, 30, 60])
def test_a_large_value_scale_of_a_low_scoring_row(dev, D, H, G, bs, where, bits):
    """One row with next to no weight, whose V scale is 2^bits that of the
    others: the others keep their precision, in its tile and in all others."""
    lens = [700]
    w, spec, pool = _case(dev, "i8", H, D, bs, lens, 101, offsets=False)
    q = rand_rows((1, H * G, D), "bf16", 102, dev).abs_()
    nb = -(-lens[0] // bs)
    at = {"first": 1, "middle": 333, "last": 690}[where]
    blk, row = int(w.batch.block_tables[0, at // bs]), at % bs
    pool.k_cache[blk, w.layer, row, :H * D] = 1           # codes -127 against positive queries:
    _scales(pool.k_cache, spec)[blk, w.layer, row] = 0.25  # its logits are the lowest by far
    _scales(pool.v_cache, spec)[blk, w.layer, row] *= 2.0 ** bits
    sel = np.tile(np.arange(nb, dtype=np.int32), (1, H, 1))
    out = torch.empty_like(q)
    bt, _, offs, _ = dev_batch(w.batch, dev)
    scale = D ** -0.5
    seq, pos = np.array([0]), np.array([lens[0] - 1])
    pkv.decode_attention_sparse(pool, w.layer, q, scale, bt, offs, _t(seq, dev), _t(pos, dev),
                                _t(sel, dev), out)
    assert pkv.device_error() == "PKV_OK"
    _check(out, q, pool, w, spec, seq, pos, sel, scale)


@pytest.mark.parametrize("D,H,G,bs", [(128, 2, 4, 16), (64, 2, 9, 8)])
@pytest.mark.parametrize("lo,hi", [(-20, 20), (-100, -60), (60, 100), (-40, 0)])
def test_value_scales_of_a_wide_range(dev, D, H, G, bs, lo, hi):
    """V scales spread over many powers of two, zeros among them."""
    lens = [400, 37, 1]
    w, spec, pool = _case(dev, "i8", H, D, bs, lens, 111)
    rng = np.random.default_rng(112)
    s = _scales(pool.v_cache, spec)
    s *= torch.exp2(torch.from_numpy(rng.uniform(lo, hi, tuple(s.shape)).astype(np.float32))).to(dev)
    s[torch.from_numpy(rng.random(tuple(s.shape)) < 0.1).to(dev)] = 0.0
    seq, pos = _queries(rng, lens, 3)
    sel = _entries(rng, seq, pos, w, H, 12, bs)
    q = rand_rows((len(seq), H * G, D), "bf16", 113, dev)
    out = torch.empty_like(q)
    bt, _, offs, _ = dev_batch(w.batch, dev)
    pkv.decode_attention_sparse(pool, w.layer, q, D ** -0.5, bt, offs, _t(seq, dev), _t(pos, dev),
                                _t(sel, dev), out)
    _check(out, q, pool, w, spec, seq, pos, sel, D ** -0.5)


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_infinite_and_negative_value_scales(dev, sign):
    """A seen row with an infinite scale gives its codes' signs times infinity and
    NaN for codes of zero; scales below zero are factors like any other."""
    D, H, G, bs = 64, 1, 4, 16
    w, spec, pool = _case(dev, "i8", H, D, bs, [90], 121, offsets=False)
    rng = np.random.default_rng(122)
    s = _scales(pool.v_cache, spec)
    s *= torch.from_numpy(rng.choice([-1.0, 1.0], tuple(s.shape)).astype(np.float32)).to(dev)
    q = rand_rows((1, G, D), "bf16", 123, dev)
    seq, pos = np.array([0]), np.array([89])
    sel = np.arange(6, dtype=np.int32).reshape(1, 1, 6)
    out = torch.empty_like(q)
    bt, _, offs, _ = dev_batch(w.batch, dev)

    def run():
        pkv.decode_attention_sparse(pool, w.layer, q, D ** -0.5, bt, offs, _t(seq, dev),
                                    _t(pos, dev), _t(sel, dev), out)

    run()
    _check(out, q, pool, w, spec, seq, pos, sel, D ** -0.5)
    blk = int(w.batch.block_tables[0, 2])
    s[blk, w.layer, 3, 0] = sign * float("inf")
    run()
    codes = pool.v_cache[blk, w.layer, 3, :D].float() - 128
    got, zero = out[0].float(), codes == 0
    assert bool(got[:, zero].isnan().all())
    assert torch.equal(got[:, ~zero], (codes.sign() * sign * float("inf"))[~zero].expand(G, -1))


@pytest.mark.parametrize("poison", [float("nan"), float("inf"), 2.0 ** 60])
@pytest.mark.parametrize("H,G,D,bs,lens,K", [
    (8, 4, 128, 16, [300, 1, 17], 9), (2, 16, 64, 8, [120], 11), (1, 10, 128, 32, [400], 8),
    (5, 2, 128, 1, [30], 13), (3, 3, 64, 64, [200, 65], 3),
])
def test_rows_that_no_query_sees(dev, H, G, D, bs, lens, K, poison):
    """Scales of other layers, of rows before an offset and past a query, and of
    blocks of no sequence are not read."""
    w, spec, pool = _case(dev, "i8", H, D, bs, lens, 131)
    rng = np.random.default_rng(132)
    seq, pos = _queries(rng, lens, 2)
    sel = _entries(rng, seq, pos, w, H, K, bs)
    seen = torch.zeros(pool.k_cache.shape[:3], dtype=torch.bool, device=dev)
    for t in range(len(seq)):
        if seq[t] >= 0:
            p = int(w.batch.offsets[seq[t]]) + np.arange(pos[t] + 1)
            seen[_t(w.batch.block_tables[seq[t]][p // bs], dev).long(), w.layer,
                 _t(p % bs, dev).long()] = True
    for c in (pool.k_cache, pool.v_cache):
        _scales(c, spec).masked_fill_(~seen[..., None], poison)
    q = rand_rows((len(seq), H * G, D), "bf16", 133, dev)
    out = torch.zeros_like(q)
    bt, _, offs, _ = dev_batch(w.batch, dev)
    pkv.decode_attention_sparse(pool, w.layer, q, D ** -0.5, bt, offs, _t(seq, dev), _t(pos, dev),
                                _t(sel, dev), out)
    # the oracle reads seen rows alone; keep the poison out of its other products
    for c in (pool.k_cache, pool.v_cache):
        _scales(c, spec).masked_fill_(~seen[..., None], 0.0)
    _check(out, q, pool, w, spec, seq, pos, sel, D ** -0.5)
    assert pkv.device_error() == "PKV_OK"
