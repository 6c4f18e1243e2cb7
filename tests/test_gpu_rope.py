"""GPU parity of the rotary append (pkv_rope_append) against the oracle in 64
bits.

Tolerances.  The kernel computes in fp32 and rounds once.  Its angle, as a
fraction of a half turn in [-1, 1), is off by 2^-25 (the conversion to fp32),
pi 2^-25 radians, sincospif by 2 units of 2^-24, and the two products and
their sum by 3 more: together less than 2^-21 (|a| + |b|) for a pair (a, b)
of attn_scale <= 1.4.  The output's rounding adds half a step, eps / 2 of the
value."""

import numpy as np
import pytest
import torch

import oracle
from oracle import quant as Q
from oracle import rope as R
import paged_kv_cache_blk_gb300 as pkv
from workloads import PoolSpec, fill_pool, fill_pool_i8, new_pool, rand_rows, small_workload
from workloads import to_numpy_bits

from gpu_util import dev_batch, need_gpu, widen_out

pytestmark = pytest.mark.gpu

BASE = 500000.0


@pytest.fixture(scope="module")
def dev():
    d = need_gpu()
    pkv.set_validate(False)
    pkv.device_error(clear=True)
    return d


def _make_pool(spec, layer, seed, dev):
    if spec.dtype == "i8":
        k = torch.zeros(spec.shape, dtype=torch.uint8, device=dev)
        v = torch.zeros_like(k)
        fill_pool_i8(k, v, spec, layer, seed)
        return pkv.Pool(k, v, spec.num_kv_heads, spec.head_dim)
    k, v = new_pool(spec, dev)
    fill_pool(k, v, spec, layer, seed)
    return pkv.Pool(k, v)


def _io(dtype):
    return "f32" if dtype == "f32" else "bf16"


def _half_step(dtype):
    return torch.finfo(torch.float32 if dtype == "f32" else torch.bfloat16).eps / 2


def _mates(x, rd, interleaved):
    """|a| + |b| of the pair each element belongs to (0 where it passes)."""
    n = np.abs(x)
    out = np.zeros_like(n)
    h = rd // 2
    ia, ib = (np.arange(0, rd, 2), np.arange(1, rd, 2)) if interleaved else (np.arange(h),
                                                                            np.arange(h, rd))
    out[..., ia] = out[..., ib] = n[..., ia] + n[..., ib]
    return out


def _check(got, x, pos, rope, freq, rd, inter, half):
    ref = R.rotate(x, pos, freq, inter, rope.attn_scale)
    tol = half * np.abs(ref) * 1.001 + 2.0 ** -21 * _mates(x, rd, inter)
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (int(bad.sum()), float(np.max(np.abs(got - ref) - tol)))
    assert np.array_equal(got[..., rd:], x[..., rd:].astype(got.dtype))


def _tokens(w, rng, pad_frac=0.15):
    seq, pos = w.tokens.token_seq.copy(), w.tokens.token_pos.copy()
    order = rng.permutation(len(seq))
    seq, pos = seq[order], pos[order]
    seq[rng.random(len(seq)) < pad_frac] = -1
    return seq.astype(np.int32), pos.astype(np.int32)


def _run(dev, dtype, H, G, D, rd, inter, bs=16, lens=None, fused=True, in_place=False,
         rope_pos=None, seed=3, **rope_kw):
    """One call on a ragged batch with padding; everything checked: q, keys and
    values at their slots, the slots, and the rest of the pool untouched."""
    w = small_workload(seed=seed, num_blocks=160, batch=4, max_len=90, num_kv_heads=H, head_dim=D,
                       dtype=_io(dtype), block_size=bs, lens=lens)
    spec = PoolSpec(160, 2, bs, H, D, dtype)
    pool = _make_pool(spec, w.layer, seed + 1, dev)
    kh, vh = to_numpy_bits(pool.k_cache), to_numpy_bits(pool.v_cache)
    rng = np.random.default_rng(seed + 2)
    seq, pos = _tokens(w, rng)
    T, hq, io = len(seq), H * G, _io(dtype)
    if fused:
        qkv = rand_rows((T, hq + 2 * H, D), io, seed + 3, dev)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + H], qkv[:, hq + H:]
    else:
        q, k, v = (rand_rows((T, h, D), io, seed + 3 + i, dev) for i, h in enumerate((hq, H, H)))
    rope = pkv.Rope(rd, base=BASE, interleaved=inter, **rope_kw)
    freq = R.inv_freq(rd, BASE, **rope_kw)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)
    rp = None if rope_pos is None else rope_pos(rng, T).astype(np.int32)
    angle_pos = pos if rp is None else rp
    xq, xk = widen_out(q), widen_out(k)
    vbits = to_numpy_bits(v)
    out = q if in_place else torch.full((T, hq, D), 7.0, dtype=q.dtype, device=dev)
    slots = torch.full((T,), -7, dtype=torch.int64, device=dev)
    bt, _, offs, _ = dev_batch(w.batch, dev)
    pkv.rope_append(pool, w.layer, rope, bt, offs, t(seq), t(pos), q, k, v, out,
                    rope_pos=None if rp is None else t(rp), slot_mapping=slots)
    torch.cuda.synchronize()
    assert pkv.device_error() == "PKV_OK"
    ref_sm = oracle.build_slot_mapping(w.batch.block_tables, w.batch.offsets, seq, pos, bs)
    assert np.array_equal(slots.cpu().numpy(), ref_sm)
    live = seq >= 0
    got = widen_out(out)
    _check(got[live], xq[live], angle_pos[live], rope, freq, rd, inter, _half_step(dtype))
    assert np.array_equal(got[~live], xq[~live] if in_place else np.full_like(got[~live], 7.0))
    blk, row = ref_sm[live] // bs, ref_sm[live] % bs
    k2, v2 = to_numpy_bits(pool.k_cache), to_numpy_bits(pool.v_cache)
    if dtype != "i8":
        keys = widen_out(pool.k_cache)[blk, w.layer, row]
        _check(keys, xk[live], angle_pos[live], rope, freq, rd, inter, _half_step(dtype))
        oracle.write_slots(kh, vh, w.layer, to_numpy_bits(k), vbits, ref_sm)
    else:
        ref = R.rotate(xk[live], angle_pos[live], freq, inter, rope.attn_scale)
        err = 2.0 ** -21 * _mates(xk[live], rd, inter)
        codes, scales = Q.unpack_rows(k2[blk, w.layer, row], H, D)
        top = np.abs(ref).max(-1)
        # the scale is absmax / 127, rounded, of fp32 values within err of ref
        assert np.all(np.abs(scales - top / 127) <= 2 * (err.max(-1) / 127 + top / 127 * 2 ** -23))
        step = scales[..., None].astype(np.float64)
        assert np.all(np.abs(codes * step - ref) <= step / 2 * (1 + 2 ** -15) + 2 * err)
        Q.write_slots_i8(kh, vh, w.layer, to_numpy_bits(k), vbits, ref_sm, H, D)
    # the values, and whatever no token of the call names, bit for bit
    assert np.array_equal(v2, vh)
    k2[blk, w.layer, row] = 0
    kh[blk, w.layer, row] = 0
    assert np.array_equal(k2, kh)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype,H,G,D,rd", [
    ("bf16", 8, 4, 128, 128), ("bf16", 2, 1, 64, 64), ("bf16", 1, 7, 128, 64),
    ("bf16", 4, 2, 32, 16), ("bf16", 3, 2, 256, 64), ("f32", 4, 3, 64, 64),
    ("f32", 2, 2, 128, 32), ("f32", 1, 5, 256, 256), ("f32", 2, 1, 32, 32),
    ("bf16", 2, 2, 128, 24), ("bf16", 2, 2, 256, 200), ("f32", 2, 2, 64, 20), ("f32", 1, 2, 256, 40),
    ("i8", 8, 4, 128, 128), ("i8", 2, 3, 64, 32), ("i8", 2, 2, 128, 72), ("i8", 4, 1, 32, 32), ("i8", 1, 2, 256, 128),
])
def test_rope_append(dev, dtype, H, G, D, rd, inter):
    _run(dev, dtype, H, G, D, rd, inter)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "i8"])
def test_contiguous_and_in_place(dev, dtype):
    _run(dev, dtype, 2, 4, 64, 64, False, fused=False, seed=11)
    _run(dev, dtype, 2, 4, 64, 32, False, in_place=True, seed=12)
    _run(dev, dtype, 2, 4, 64, 32, True, in_place=True, fused=False, seed=13)


@pytest.mark.parametrize("kw", [dict(scaling="linear", factor=8.0),
                                dict(scaling="base", factor=4.0),
                                dict(scaling="by_parts", factor=16.0, original_len=4096)])
def test_long_context_schedules(dev, kw):
    _run(dev, "f32", 2, 2, 128, 128, False, seed=21, **kw)


@pytest.mark.parametrize("lo,hi", [(-(1 << 31), 1 << 31), (1 << 20, 1 << 21), (-5, 5)])
def test_rotary_positions_of_their_own(dev, lo, hi):
    """Any 32-bit position: the angle is exact modulo one turn."""
    _run(dev, "f32", 2, 2, 64, 64, True, seed=31, rope_pos=lambda r, n: r.integers(lo, hi, n))


@pytest.mark.parametrize("bs,lens", [(1, [1, 0, 7]), (16, [1]), (64, [130, 64, 1, 65]),
                                     (1024, [1500])])
def test_block_sizes_and_one_token(dev, bs, lens):
    _run(dev, "bf16", 4, 4, 128, 128, False, bs=bs, lens=lens, seed=41)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "i8"])
def test_position_zero_is_append_tokens(dev, dtype):
    """At rotary position 0 nothing turns: the pool holds what append_tokens stores."""
    H, D, T = 4, 128, 37
    w = small_workload(seed=51, num_blocks=64, lens=[T], num_kv_heads=H, head_dim=D,
                       dtype=_io(dtype))
    spec = PoolSpec(64, 2, 16, H, D, dtype)
    a, b = (_make_pool(spec, 1, 52, dev) for _ in range(2))
    bt, _, offs, _ = dev_batch(w.batch, dev)
    seq = torch.zeros(T, dtype=torch.int32, device=dev)
    pos = torch.arange(T, dtype=torch.int32, device=dev)
    k, v = rand_rows((T, H, D), _io(dtype), 53, dev), rand_rows((T, H, D), _io(dtype), 54, dev)
    pkv.append_tokens(a, 1, bt, offs, seq, pos, k, v)
    pkv.rope_append(b, 1, pkv.Rope(D), bt, offs, seq, pos, None, k, v, None,
                    rope_pos=torch.zeros_like(pos))
    assert torch.equal(a.k_cache, b.k_cache) and torch.equal(a.v_cache, b.v_cache)


def test_bad_tokens_are_skipped_and_reported(dev):
    w = small_workload(seed=61, num_blocks=48, batch=3, lens=[40, 20, 33])
    pool = _make_pool(w.pool, w.layer, 62, dev)
    before = (pool.k_cache.clone(), pool.v_cache.clone())
    H, D = w.pool.num_kv_heads, w.pool.head_dim
    cap = int(w.batch.block_tables.shape[1]) * w.pool.block_size
    t = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)
    k, q = rand_rows((4, H, D), "bf16", 63, dev), rand_rows((4, 4, D), "bf16", 64, dev)
    out = torch.full_like(q, 7.0)
    bt, _, offs, _ = dev_batch(w.batch, dev)
    args = (pool, w.layer, pkv.Rope(D), bt, offs, t([3, 0, -1, 1]), t([0, cap, 5, -1]), q, k, k, out)
    pkv.rope_append(*args)
    assert pkv.device_error() in ("PKV_ERR_INDEX", "PKV_ERR_CAPACITY")
    assert torch.equal(out, torch.full_like(out, 7.0))
    assert torch.equal(pool.k_cache, before[0]) and torch.equal(pool.v_cache, before[1])
    pkv.set_validate(True)
    try:
        with pytest.raises(pkv.PkvError):
            pkv.rope_append(*args)
    finally:
        pkv.set_validate(False)
    assert pkv.device_error() == "PKV_OK"


def test_binding_refusals(dev):
    w = small_workload(seed=71, num_blocks=16, lens=[20])
    pool = _make_pool(w.pool, w.layer, 72, dev)
    H, D, T = w.pool.num_kv_heads, w.pool.head_dim, 20
    bt, _, offs, _ = dev_batch(w.batch, dev)
    seq = torch.zeros(T, dtype=torch.int32, device=dev)
    pos = torch.arange(T, dtype=torch.int32, device=dev)
    k = rand_rows((T, H, D), "bf16", 73, dev)
    rope = pkv.Rope(D)

    def call(**kw):
        a = dict(bt=bt, offs=offs, seq=seq, pos=pos, q=k, k=k, v=k, out=torch.empty_like(k))
        a.update(kw)
        pkv.rope_append(pool, 0, rope, *a.values())

    call()
    for kw in (dict(seq=seq.long()), dict(pos=pos[:-1]), dict(bt=bt.cpu()), dict(k=k.float()),
               dict(v=k[:, :1]), dict(q=k[:-1]), dict(out=None), dict(q=k.transpose(1, 2)),
               dict(out=k[..., :32]), dict(offs=offs.repeat(2)), dict(pos=pos.flip(0)[::1][::2]),
               dict(q=torch.empty((T, D, H), dtype=k.dtype, device=dev).transpose(1, 2))):
        with pytest.raises(ValueError):
            call(**kw)


def test_graph_replay_and_another_stream(dev):
    """A captured call replayed on new inputs gives what an eager one gives."""
    H, D, T = 2, 128, 5
    w = small_workload(seed=81, num_blocks=64, lens=[30, 60, 12, 90, 1], num_kv_heads=H, head_dim=D,
                       num_layers=1, layer=0)
    pools = [_make_pool(w.pool, 0, 82, dev) for _ in range(2)]
    bt, lens, offs, _ = dev_batch(w.batch, dev)
    seq = torch.arange(T, dtype=torch.int32, device=dev)
    pos = (lens - 1).to(torch.int32)
    rope = pkv.Rope(D, base=BASE)
    q, k, v = (rand_rows((T, h, D), "bf16", 83 + h, dev) for h in (8, H, H))
    outs = [torch.zeros_like(q) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pkv.rope_append(pools[0], 0, rope, bt, offs, seq, pos, q, k, v, outs[0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.rope_append(pools[0], 0, rope, bt, offs, seq, pos, q, k, v, outs[0])
    for step in range(3):
        q.copy_(rand_rows(q.shape, "bf16", 90 + step, dev))
        k.copy_(rand_rows(k.shape, "bf16", 95 + step, dev))
        pos.sub_(pos.clamp(max=1))
        g.replay()
        pkv.rope_append(pools[1], 0, rope, bt, offs, seq, pos, q, k, v, outs[1])
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1])
    # the first position was written in pool 0 only by the eager call: rewrite it in pool 1
    pos.copy_(lens - 1)
    pkv.rope_append(pools[0], 0, rope, bt, offs, seq, pos, q, k, v, outs[0])
    pkv.rope_append(pools[1], 0, rope, bt, offs, seq, pos, q, k, v, outs[1])
    torch.cuda.synchronize()
    assert torch.equal(pools[0].k_cache, pools[1].k_cache)
    assert torch.equal(pools[0].v_cache, pools[1].v_cache)
