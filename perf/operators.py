"""Timed cases of the rotary append and of sparse decode over the paged cache.

Four operators, in the order in which a decode step of a server with long
contexts uses them:

``rope_append``   rotary positions on q and on the new keys, the rotated keys
                  and the values stored at their slots (``pkv.rope_append``);
``bounds``        per-block key bounds of the blocks that hold new tokens
                  (``pkv.update_block_bounds``);
``select``        score of every block of a query's sequence from those
                  bounds, and the best blocks (``pkv.select_blocks``);
``sparse``        attention over the selected blocks
                  (``pkv.decode_attention_sparse``).

With ``own`` false ``run`` computes them with elementary torch operations, with
``own`` true through the library.  ``exact`` is the definition in 64 bits.
"""

import math
import zlib
from types import SimpleNamespace

import numpy as np
import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32, "i8": torch.bfloat16}  # of q and of new rows
BASE = 500000.0      # rotary base
E_MIN, E_MAX = -40, 40  # range of the exponents of 8-bit codes with power-of-two scales


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one user decoding at the end of a long context: nothing but latency
        dict(name="rope_one_token", op="rope_append", dtype="bf16", hq=32, hkv=8, d=128, bs=16, layers=1,
             seqs=1, tokens=1, pad=0.0, start=131071, rd=128, interleaved=False, fused=False, offsets=False),
        # a batch of prompts of 8192 entries with a tenth of padding, q, k and v in
        # one projection's output, half of each head rotated in adjacent pairs
        dict(name="rope_prompts_8192", op="rope_append", dtype="bf16", hq=32, hkv=8, d=128, bs=16, layers=1,
             seqs=8, tokens=8192, pad=0.1, start=0, rd=64, interleaved=True, fused=True, offsets=True),
        # chunks of prompts after a cached context into an int8 pool
        dict(name="rope_chunks_i8", op="rope_append", dtype="i8", hq=32, hkv=8, d=128, bs=16, layers=1,
             seqs=16, tokens=6000, pad=0.0, start=20000, rd=128, interleaved=False, fused=True, offsets=False),
        # after prompts were stored: the bounds of all their blocks
        dict(name="bounds_prompts", op="bounds", dtype="bf16", hkv=8, d=128, bs=16, layers=1,
             seqs=32, len_lo=512, len_hi=4096, tail=0, offsets=True),
        # one short sequence in an int8 pool
        dict(name="bounds_short_i8", op="bounds", dtype="i8", hkv=4, d=64, bs=16, layers=1,
             seqs=1, len_lo=100, len_hi=100, tail=0, offsets=False),
        # one user, 131072 tokens of context, 2048 of them to be read
        dict(name="select_one_131072", op="select", dtype="bf16", hq=32, hkv=8, d=128, bs=16, layers=1,
             seqs=1, queries=1, len_lo=131072, len_hi=131072, k=128, sink=1, recent=4, offsets=False),
        # an ordinary decode batch, two layers in the pool
        dict(name="select_batch_64", op="select", dtype="bf16", hq=32, hkv=8, d=128, bs=16, layers=2,
             seqs=64, queries=1, len_lo=1024, len_hi=8192, k=64, sink=2, recent=2, offsets=True),
        # a few very long sequences, three tokens each being verified, fp32
        dict(name="select_long_verify", op="select", dtype="f32", hq=20, hkv=4, d=64, bs=16, layers=1,
             seqs=8, queries=3, len_lo=32768, len_hi=131072, k=300, sink=1, recent=1, offsets=True),
        # one user, 64 blocks selected: latency
        dict(name="sparse_one_64", op="sparse", dtype="bf16", hq=32, hkv=8, d=128, bs=16, layers=1,
             seqs=1, queries=1, len_lo=16384, len_hi=16384, k=64, offsets=False),
        # an ordinary decode batch that reads 2048 tokens a head
        dict(name="sparse_batch_64", op="sparse", dtype="bf16", hq=32, hkv=8, d=128, bs=16, layers=1,
             seqs=64, queries=1, len_lo=1024, len_hi=8192, k=128, offsets=True),
        # the same from an int8 pool
        dict(name="sparse_batch_64_i8", op="sparse", dtype="i8", hq=32, hkv=8, d=128, bs=16, layers=1,
             seqs=64, queries=1, len_lo=1024, len_hi=8192, k=128, offsets=True),
        # fp32, three query heads a kv head, several queries a sequence, few blocks of 32 rows
        dict(name="sparse_verify_f32", op="sparse", dtype="f32", hq=12, hkv=4, d=64, bs=32, layers=2,
             seqs=13, queries=3, len_lo=1, len_hi=3000, k=17, offsets=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope_append", "bounds", "select", "sparse"])
    dtype = rng.choice(["bf16", "bf16", "i8", "f32"])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8, 8])
    group = rng.choice([1, 2, 3, 4, 4, 5, 8, 16])
    bs = rng.choice([8, 16, 16, 32, 64])
    c = dict(op=op, dtype=dtype, hkv=hkv, d=d, bs=bs, layers=rng.choice([1, 2]), offsets=rng.random() < 0.5)
    if op == "rope_append":
        group = min(group, 8)
        tokens = _log(rng, 1, 6000)
        c.update(hq=hkv * group, tokens=tokens, seqs=min(tokens, _log(rng, 1, 64)), pad=rng.choice([0.0, 0.1]),
                 start=_log(rng, 1, 1 << 20) - 1, rd=rng.choice([32, 64, d]), interleaved=rng.random() < 0.5,
                 fused=rng.random() < 0.5)
        if c["seqs"] == tokens:
            c["pad"] = 0.0
    elif op == "bounds":
        hi = _log(rng, 30, 4096)
        c.update(seqs=_log(rng, 1, 24), len_lo=max(1, hi // 8), len_hi=hi, tail=rng.choice([0, 0, 1, 40]))
    elif op == "select":
        hi = _log(rng, 100, 65536)
        seqs = max(1, min(_log(rng, 1, 64), 262144 // hi))
        k = _log(rng, 8, 400)
        c.update(hq=hkv * group, seqs=seqs, queries=rng.choice([1, 1, 2, 5]), len_lo=max(1, hi // 8), len_hi=hi, k=k,
                 sink=rng.randint(0, 2), recent=rng.randint(0, 4))
    else:
        hi = _log(rng, 100, 16384)
        seqs = _log(rng, 1, 48)
        queries = rng.choice([1, 1, 2, 5]) if seqs <= 12 else 1
        k = max(1, min(_log(rng, 4, 256), (60000 if dtype == "f32" else 120000) // (bs * seqs * queries)))
        c.update(hq=hkv * group, seqs=seqs, queries=queries, len_lo=max(1, hi // 8), len_hi=hi, k=k)
    return c


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _row_bytes(c):
    return c["hkv"] * c["d"] + (4 * c["hkv"] + 15) // 16 * 16


def _new_pool(c, n, gen, fill):
    """K or V cache of ``n`` blocks: N(0, 1) rows, or int8 codes and scales of such rows."""
    H, D = c["hkv"], c["d"]
    if c["dtype"] != "i8":
        shape = (n, c["layers"], c["bs"], H, D)
        if not fill:
            return torch.zeros(shape, dtype=DTYPE[c["dtype"]], device="cuda")
        return torch.randn(shape, generator=gen, device="cuda", dtype=DTYPE[c["dtype"]])
    p = torch.zeros((n, c["layers"], c["bs"], _row_bytes(c)), dtype=torch.uint8, device="cuda")
    if fill:
        codes = (torch.randn(p.shape[:3] + (H * D,), generator=gen, device="cuda") * 42).round_().clamp_(-127, 127)
        p[..., :H * D] = (codes + 128).to(torch.uint8)
        scales = torch.rand(p.shape[:3] + (H,), generator=gen, device="cuda") * 0.03 + 0.01
        p[..., H * D:H * D + 4 * H] = scales.view(torch.uint8).view(p.shape[:3] + (4 * H,))
    return p


def _cuda(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dtype)


def _shapes(c):
    """The lengths, offsets and starts of a case are the same multiset for every seed, so that a case has one size of
    cache and one amount of work; a seed gives their order."""
    return np.random.RandomState(zlib.crc32(repr(sorted((k, v) for k, v in c.items() if k != "name")).encode()))


def _lengths(c):
    f = _shapes(c)
    lens = f.randint(c["len_lo"], c["len_hi"] + 1, c["seqs"])
    return lens, f.randint(0, c["bs"], c["seqs"]) if c["offsets"] else np.zeros(c["seqs"], np.int64)


def _sequences(c, r):
    """Lengths, first-block offsets and block tables of ragged sequences, every block a sequence's own."""
    bs, B = c["bs"], c["seqs"]
    order = r.permutation(B)
    lens, offs = (x[order] for x in _lengths(c))
    nblk = -(-(offs + lens) // bs)
    n = int(nblk.sum())
    ids = r.permutation(n)
    table = np.full((B, int(nblk.max())), -1, np.int64)
    at = 0
    for b in range(B):
        table[b, :nblk[b]] = ids[at:at + nblk[b]]
        at += nblk[b]
    return lens, offs, table, n


def _tokens(c, lens):
    """The last ``queries`` positions of each sequence (fewer where it is shorter: the others are padding)."""
    q = c["queries"]
    seq = np.repeat(np.arange(len(lens)), q)
    pos = (lens[:, None] - q + np.arange(q)[None]).reshape(-1)
    return np.where(pos >= 0, seq, -1), np.maximum(pos, 0)


def prepare(case, seed):
    c = case
    r = np.random.RandomState(seed % (1 << 31))
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = SimpleNamespace(case=c, op=c["op"], layer=c["layers"] - 1)
    return {"rope_append": _prepare_rope, "bounds": _prepare_bounds, "select": _prepare_select,
            "sparse": _prepare_sparse}[c["op"]](s, c, r, gen)


def _handle(s, c, k, v):
    """What a program keeps of its cache: with the library, its pool descriptor too."""
    s.k, s.v = k, v
    if own:
        import paged_kv_cache_blk_gb300 as pkv
        s.pkv = pkv
        s.pool = pkv.Pool(k, v, c["hkv"], c["d"]) if c["dtype"] == "i8" else pkv.Pool(k, v)


def _inv_freq(c):
    """Rotary frequencies, base ** (-2 i / rd)."""
    return BASE ** (-np.arange(0, c["rd"], 2, dtype=np.float64) / c["rd"])


def _prepare_rope(s, c, r, gen):
    B, T, bs, H, D, Hq = c["seqs"], c["tokens"], c["bs"], c["hkv"], c["d"], c["hq"]
    n = max(B, T - int(T * c["pad"]))
    pad = np.zeros(T, bool)
    pad[r.permutation(T)[n:]] = True
    f, order = _shapes(c), r.permutation(B)
    cuts = np.sort(f.choice(np.arange(1, n), B - 1, replace=False)) if B > 1 else np.zeros(0, np.int64)
    count = np.diff(np.concatenate([[0], cuts, [n]]))[order]
    start = (f.randint(0, c["start"] + 1, B) if B > 1 else np.array([c["start"]]))[order]
    offs = (f.randint(0, bs, B) if c["offsets"] else np.zeros(B, np.int64))[order]
    first, last = (offs + start) // bs, (offs + start + count - 1) // bs
    nblk = int((last - first + 1).sum())
    ids, table, at = r.permutation(nblk), np.zeros((B, int(last.max()) + 1), np.int64), 0
    for b in range(B):
        w = last[b] - first[b] + 1
        table[b, first[b]:last[b] + 1] = ids[at:at + w]
        at += w
    seq, pos = np.full(T, -1), np.zeros(T, np.int64)
    seq[~pad] = np.repeat(np.arange(B), count)
    pos[~pad] = np.concatenate([start[b] + np.arange(count[b]) for b in range(B)])
    s.table, s.offs, s.seq, s.pos = _cuda(table), _cuda(offs), _cuda(seq), _cuda(pos)
    dt = DTYPE[c["dtype"]]
    if c["fused"]:
        qkv = torch.randn((T, Hq + 2 * H, D), generator=gen, device="cuda", dtype=dt)
        s.q, s.k_new, s.v_new = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
    else:
        s.q, s.k_new, s.v_new = (torch.randn((T, h, D), generator=gen, device="cuda", dtype=dt) for h in (Hq, H, H))
    s.q_out = torch.zeros((T, Hq, D), dtype=dt, device="cuda")
    s.inv_freq = torch.from_numpy(_inv_freq(c)).cuda()
    _handle(s, c, _new_pool(c, nblk, gen, False), _new_pool(c, nblk, gen, False))
    if own:
        s.rope = s.pkv.Rope(c["rd"], base=BASE, interleaved=c["interleaved"])
    return s


def _prepare_bounds(s, c, r, gen):
    lens, offs, table, n = _sequences(c, r)
    s.lens, s.offs, s.table = _cuda(lens), _cuda(offs), _cuda(table)
    s.first = _cuda(np.maximum(0, lens - c["tail"])) if c["tail"] else None
    k = _new_pool(c, n, gen, True)
    _handle(s, c, k, torch.zeros_like(k))
    s.codes = torch.full((n, c["layers"], c["hkv"], 2, c["d"]), 128, dtype=torch.uint8, device="cuda")
    s.scales = torch.zeros((n, c["layers"], c["hkv"]), dtype=torch.float32, device="cuda")
    if own:
        s.bounds = s.pkv.BlockBounds(s.codes, s.scales)
    return s


def _prepare_select(s, c, r, gen):
    H, D = c["hkv"], c["d"]
    lens, offs, table, n = _sequences(c, r)
    seq, pos = _tokens(c, lens)
    s.offs, s.table, s.seq, s.pos = _cuda(offs), _cuda(table), _cuda(seq), _cuda(pos)
    s.q = torch.randn((len(seq), c["hq"], D), generator=gen, device="cuda", dtype=DTYPE[c["dtype"]])
    # bounds of blocks of N(0, 1) keys around a mean of each head and dimension: the largest of 16 such keys
    # lies near 1.8 +- 0.5
    mean = torch.randn((H, D), generator=gen, device="cuda") * 0.5
    shape = (n, c["layers"], H, D)
    hi = mean + (torch.randn(shape, generator=gen, device="cuda") * 0.5 + 1.8).clamp_(0.1)
    lo = mean - (torch.randn(shape, generator=gen, device="cuda") * 0.5 + 1.8).clamp_(0.1)
    s.codes = (torch.stack([(hi * 24).ceil_(), (lo * 24).floor_()], 3).clamp_(-127, 127) + 128).to(torch.uint8)
    s.scales = torch.exp2(torch.randint(-5, -3, shape[:3], generator=gen, device="cuda").float())
    k = torch.zeros((n, c["layers"], c["bs"], _row_bytes(c)), dtype=torch.uint8, device="cuda") \
        if c["dtype"] == "i8" else torch.zeros((n, c["layers"], c["bs"], H, D), dtype=DTYPE[c["dtype"]], device="cuda")
    _handle(s, c, k, k)
    s.sel = torch.empty((len(seq), H, c["k"]), dtype=torch.int32, device="cuda")
    s.count = torch.empty((len(seq), H), dtype=torch.int32, device="cuda")
    if own:
        s.bounds = s.pkv.BlockBounds(s.codes, s.scales)
    return s


def _prepare_sparse(s, c, r, gen):
    H = c["hkv"]
    lens, offs, table, n = _sequences(c, r)
    seq, pos = _tokens(c, lens)
    s.offs, s.table, s.seq, s.pos = _cuda(offs), _cuda(table), _cuda(seq), _cuda(pos)
    s.scale = c["d"] ** -0.5
    s.q = torch.randn((len(seq), c["hq"], c["d"]), generator=gen, device="cuda", dtype=DTYPE[c["dtype"]])
    _handle(s, c, _new_pool(c, n, gen, True), _new_pool(c, n, gen, True))
    # for each head the first block, the last one and random ones between, ascending, -1 behind
    sel = np.full((len(seq), H, c["k"]), -1, np.int64)
    for t in range(len(seq)):
        if seq[t] < 0:
            continue
        nb = int((offs[seq[t]] + pos[t]) // c["bs"]) + 1
        for g in range(H):
            if nb <= c["k"]:
                sel[t, g, :nb] = np.arange(nb)
                continue
            keep = r.choice(nb - 1, c["k"] - 1, replace=False)
            if c["k"] > 1 and 0 not in keep:
                keep[0] = 0
            sel[t, g, :c["k"]] = np.sort(np.append(keep, nb - 1))
    s.sel = _cuda(sel)
    s.out = torch.zeros_like(s.q)
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(state):
    s = state
    if own:
        return _OWN[s.op](s)
    return _PLAIN[s.op](s)


def _own_rope(s):
    s.pkv.rope_append(s.pool, s.layer, s.rope, s.table, s.offs, s.seq, s.pos, s.q, s.k_new, s.v_new, s.q_out)
    return {"q": s.q_out, "k": _values(s, s.k), "v": _values(s, s.v)}


def _own_bounds(s):
    s.pkv.update_block_bounds(s.pool, s.layer, s.bounds, s.table, s.lens, s.offs, s.first)
    return _bound_values(s)


def _own_select(s):
    c = s.case
    s.pkv.select_blocks(s.pool, s.layer, s.bounds, s.q, s.table, s.offs, s.seq, s.pos, s.sel, s.count,
                        sink=c["sink"], recent=c["recent"])
    return {"sel": s.sel, "count": s.count}


def _own_sparse(s):
    s.pkv.decode_attention_sparse(s.pool, s.layer, s.q, s.scale, s.table, s.offs, s.seq, s.pos, s.sel, s.out)
    return s.out


def _values(s, cache):
    """What a cache holds: itself, or the numbers that int8 codes and scales stand for, in the type of the new rows."""
    c = s.case
    if c["dtype"] != "i8":
        return cache
    HD, H = c["hkv"] * c["d"], c["hkv"]
    codes = (cache[..., :HD] - 128.0).unflatten(-1, (H, c["d"]))
    scales = cache[..., HD:HD + 4 * H].view(torch.float32)[..., None]
    return torch.mul(codes, scales, out=torch.empty(codes.shape, dtype=DTYPE["i8"], device="cuda"))


def _bound_values(s):
    return (s.codes - 128.0).mul_(s.scales[..., None, None])


def _slots(s, seq, pos):
    """Physical block and row of a position of a sequence."""
    p = s.offs[seq].long() + pos
    return s.table[seq, p // s.case["bs"]].long(), p % s.case["bs"]


def _plain_rope(s):
    c = s.case
    rd, T = c["rd"], c["tokens"]
    ang = s.pos.double()[:, None] * s.inv_freq  # in 64 bits: far positions
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]

    def rotate(x):
        x = x.float()
        if c["interleaved"]:
            a, b = x[..., 0:rd:2], x[..., 1:rd:2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = x[..., :rd // 2], x[..., rd // 2:rd]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([y, x[..., rd:]], -1)

    valid = s.seq >= 0
    q = torch.where(valid[:, None, None], rotate(s.q).to(s.q.dtype), s.q_out)
    # padding entries repeat the first real one's store
    src = torch.where(valid, torch.arange(T, device="cuda"), valid.int().argmax())
    blk, row = _slots(s, s.seq[src].long(), s.pos[src].long())
    for cache, x in ((s.k, rotate(s.k_new)), (s.v, s.v_new.float())):
        x = x[src]
        if c["dtype"] != "i8":
            cache[blk, s.layer, row] = x.to(cache.dtype)
            continue
        scale = x.abs().amax(-1) / 127
        code = torch.where(scale[..., None] > 0, x / scale[..., None], 0.0).round_().clamp_(-127, 127)
        HD, H = c["hkv"] * c["d"], c["hkv"]
        cache[blk, s.layer, row, :HD] = (code + 128).to(torch.uint8).flatten(1)
        cache[blk, s.layer, row, HD:HD + 4 * H] = scale.view(torch.uint8).view(T, 4 * H)
    return {"q": q, "k": _values(s, s.k), "v": _values(s, s.v)}


def _rows(s, cache, blk, row, head=None):
    """Rows of a cache in 32 bits: all heads, or one head each."""
    c = s.case
    H, D = c["hkv"], c["d"]
    if c["dtype"] != "i8":
        return (cache[blk, s.layer, row] if head is None else cache[blk, s.layer, row, head]).float()
    codes = cache[..., :H * D].unflatten(-1, (H, D))
    scales = cache[..., H * D:H * D + 4 * H].view(torch.float32)
    if head is None:
        return (codes[blk, s.layer, row] - 128.0).mul_(scales[blk, s.layer, row][..., None])
    return (codes[blk, s.layer, row, head] - 128.0).mul_(scales[blk, s.layer, row, head][..., None])


def _exponent(absmax):
    """The smallest e in [E_MIN, E_MAX] with absmax <= 127 * 2 ** e."""
    m, x = torch.frexp(absmax)
    e = torch.where(m <= 127 / 128, x - 7, x - 6)
    return torch.where(absmax > 0, e, E_MIN).clamp_(E_MIN, E_MAX)


def _plain_bounds(s):
    c = s.case
    bs, mb = c["bs"], s.table.shape[1]
    end = s.offs + s.lens  # table positions held
    start = s.offs + (s.first if s.first is not None else 0)
    j = torch.arange(mb, device="cuda")[None]
    held = (j >= (start // bs)[:, None]) & (j * bs < end[:, None])
    # entries outside repeat the last block of their sequence
    j = torch.where(held, j, ((end - 1) // bs)[:, None])
    blk = s.table.gather(1, j.long()).long()
    row = torch.arange(bs, device="cuda")
    k = _rows(s, s.k, blk[..., None], row)  # [B, mb, bs, H, D]
    seen = ((j * bs)[..., None] + row < end[:, None, None])[..., None, None]
    hi = torch.where(seen, k, -math.inf).amax(2)
    lo = torch.where(seen, k, math.inf).amin(2)
    scale = torch.exp2(_exponent(torch.maximum(hi.abs(), lo.abs()).amax(-1)).float())
    codes = torch.stack([(hi / scale[..., None]).ceil_(), (lo / scale[..., None]).floor_()], 3).clamp_(-127, 127)
    s.codes[blk, s.layer] = (codes + 128).to(torch.uint8)
    s.scales[blk, s.layer] = scale
    return _bound_values(s)


def _plain_select(s):
    c = s.case
    H, D, K, bs, mb = c["hkv"], c["d"], c["k"], c["bs"], s.table.shape[1]
    q = s.q.float().unflatten(1, (H, -1))  # [T, H, G, D]
    qscale = torch.exp2(_exponent(q.abs().amax(-1, keepdim=True)).float())
    q = (q / qscale).round_().clamp_(-127, 127)
    valid = s.seq >= 0
    seq = s.seq.clamp(min=0).long()
    blk = s.table[seq].clamp(min=0).long()  # [T, mb]
    bound = (s.codes[blk, s.layer] - 128.0).permute(0, 2, 3, 4, 1)  # [T, H, 2, D, mb]
    # whole numbers below 2 ** 23: exact in any order
    dot = q.clamp(min=0) @ bound[:, :, 0] + q.clamp(max=0) @ bound[:, :, 1]
    score = (dot * qscale).amax(2) * s.scales[blk, s.layer].transpose(1, 2)  # [T, H, mb]
    n = torch.where(valid, (s.offs[seq] + s.pos) // bs + 1, 0)[:, None, None]  # blocks of each query
    j = torch.arange(mb, device="cuda")
    score = torch.where((j < c["sink"]) | (j >= n - c["recent"]), math.inf, score)
    score = torch.where(j < n, score, -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True)[1][..., :K]
    order = torch.where(order < n, order, mb).sort(-1)[0]
    sel = torch.where(order < mb, order, -1).int()
    if mb < K:
        sel = torch.nn.functional.pad(sel, (0, K - mb), value=-1)
    return {"sel": sel, "count": n[..., 0].clamp(max=K).int().repeat(1, H)}


def _plain_sparse(s):
    c = s.case
    T, H, K = s.sel.shape
    bs, G = c["bs"], c["hq"] // H
    seq = s.seq.clamp(min=0).long()
    j = s.sel.clamp(min=0).long()
    blk = s.table[seq[:, None, None], j].clamp(min=0).long()
    row = torch.arange(bs, device="cuda")
    p = (j * bs)[..., None] + row  # [T, H, K, bs], table positions
    off = s.offs[seq][:, None, None, None]
    seen = (p >= off) & (p <= off + s.pos[:, None, None, None]) & (s.sel >= 0)[..., None] \
        & (s.seq >= 0)[:, None, None, None]
    head = torch.arange(H, device="cuda")[:, None, None]
    k = _rows(s, s.k, blk[..., None], row, head).flatten(2, 3)  # [T, H, K * bs, D]
    q = s.q.float().unflatten(1, (H, G))
    x = (q @ k.transpose(2, 3)) * s.scale
    del k
    x = torch.where(seen.flatten(2)[:, :, None], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    w = (x - torch.where(top > -math.inf, top, 0.0)).exp_()
    total = w.sum(-1, keepdim=True)
    v = _rows(s, s.v, blk[..., None], row, head).flatten(2, 3)
    out = (w @ v) / torch.where(total > 0, total, 1.0)
    return out.flatten(1, 2).to(s.q.dtype)


_OWN = {"rope_append": _own_rope, "bounds": _own_bounds, "select": _own_select, "sparse": _own_sparse}
_PLAIN = {"rope_append": _plain_rope, "bounds": _plain_bounds, "select": _plain_select, "sparse": _plain_sparse}


# --------------------------------------------------------------------------
# the work of one pass
# --------------------------------------------------------------------------

def _kv_row(c):
    """Bytes of one head of a stored token row."""
    return {"bf16": 2, "f32": 4, "i8": 1}[c["dtype"]] * c["d"] + (4 if c["dtype"] == "i8" else 0)


def work(case):
    c = case
    io = 4 if c["dtype"] == "f32" else 2
    H, D = c["hkv"], c["d"]
    if c["op"] == "rope_append":
        n = c["tokens"] * (1 - c["pad"])
        read = n * (c["hq"] + 2 * H) * D * io
        write = n * (c["hq"] * D * io + 2 * H * _kv_row(c))
        return {"bytes": read + write, "flops": n * (c["hq"] + H) * c["rd"] * 3}
    lens, offs = _lengths(c)
    blocks = (offs + lens + c["bs"] - 1) // c["bs"]
    if c["op"] == "bounds":
        first = (offs + np.maximum(0, lens - c["tail"]) * (c["tail"] > 0)) // c["bs"]  # first block with new tokens
        rows = (offs + lens - first * c["bs"]).sum()
        return {"bytes": int(rows * H * _kv_row(c) + (blocks - first).sum() * H * (2 * D + 4)),
                "flops": int(rows * H * D * 2)}
    T = c["seqs"] * c["queries"]
    if c["op"] == "select":
        scored = int(blocks[blocks > c["k"]].sum())  # where all of them are taken, none has to be scored
        return {"bytes": scored * (H * (2 * D + 4) + 4) + T * (c["hq"] * D * io + H * c["k"] * 4),
                "flops": scored * c["queries"] * c["hq"] * D * 2}
    tokens = int(np.minimum(c["k"] * c["bs"], lens).sum()) * c["queries"]  # read for each kv head
    return {"bytes": tokens * H * 2 * _kv_row(c) + T * (2 * c["hq"] * D * io + H * c["k"] * 4),
            "flops": tokens * c["hq"] * D * 4}


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------

def _np(t):
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy().astype(np.int64)


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope_append": _exact_rope, "bounds": _exact_bounds, "select": _exact_select,
            "sparse": _exact_sparse}[case["op"]](s, case)


def _exact_head(x, pair, ang):
    """One rotation of the pairs ``pair`` (two index lists) of the last axis by ``ang``."""
    y = x.copy()
    z = (x[..., pair[0]] + 1j * x[..., pair[1]]) * np.exp(1j * ang)[:, None]
    y[..., pair[0]], y[..., pair[1]] = z.real, z.imag
    return y


def _exact_rope(s, c):
    q, k, v, seq, pos, table, offs = map(_np, (s.q, s.k_new, s.v_new, s.seq, s.pos, s.table, s.offs))
    half = np.arange(c["rd"] // 2)
    pair = (2 * half, 2 * half + 1) if c["interleaved"] else (half, half + c["rd"] // 2)
    ang = pos[:, None] * _inv_freq(c)
    q, k = _exact_head(q, pair, ang), _exact_head(k, pair, ang)
    q[seq < 0] = 0
    shape = (s.k.shape[0], c["layers"], c["bs"], c["hkv"], c["d"])
    kc, vc = np.zeros(shape), np.zeros(shape)
    for t in np.flatnonzero(seq >= 0):
        p = offs[seq[t]] + pos[t]
        at = (table[seq[t], p // c["bs"]], s.layer, p % c["bs"])
        for cache, x in ((kc, k[t]), (vc, v[t])):
            if c["dtype"] == "i8":
                # the scale of a head is defined as one division in fp32
                unit = (np.abs(x).max(-1, keepdims=True).astype(np.float32) / np.float32(127)).astype(np.float64)
                x = np.where(unit > 0, np.rint(x / np.where(unit > 0, unit, 1)), 0) * unit
            cache[at] = x
    return {"q": q, "k": kc, "v": vc}


def _exact_rows(s, c, cache):
    """A layer of a cache in 64 bits: [blocks, bs, H, D]."""
    if c["dtype"] != "i8":
        return _np(cache[:, s.layer])
    a = cache[:, s.layer].cpu().numpy()
    HD, H = c["hkv"] * c["d"], c["hkv"]
    unit = np.ascontiguousarray(a[..., HD:HD + 4 * H]).view(np.float32).astype(np.float64)
    return (a[..., :HD].reshape(a.shape[:2] + (H, c["d"])).astype(np.float64) - 128) * unit[..., None]


def _exact_exponent(top):
    e = np.full(top.shape, E_MIN)
    some = top > 0
    e[some] = np.ceil(np.log2(top[some] / 127))
    e += top > 127 * np.exp2(e.astype(np.float64))  # where the logarithm was rounded
    e -= (top <= 127 * np.exp2(e - 1.0)) & some
    return np.clip(e, E_MIN, E_MAX)


def _exact_bounds(s, c):
    rows = _exact_rows(s, c, s.k)
    table, offs, lens = map(_np, (s.table, s.offs, s.lens))
    first = _np(s.first) if s.first is not None else np.zeros_like(lens)
    got = np.zeros(tuple(s.codes.shape))
    for b in range(len(lens)):
        end = offs[b] + lens[b]
        for j in range((offs[b] + first[b]) // c["bs"], (end - 1) // c["bs"] + 1):
            x = rows[table[b, j], :end - j * c["bs"]]
            hi, lo = x.max(0), x.min(0)
            unit = np.exp2(_exact_exponent(np.maximum(abs(hi), abs(lo)).max(-1)).astype(np.float64))[:, None]
            got[table[b, j], s.layer] = np.clip(np.stack([np.ceil(hi / unit), np.floor(lo / unit)], 1),
                                                -127, 127) * unit[..., None]
    return got


def _exact_select(s, c):
    H, K, bs = c["hkv"], c["k"], c["bs"]
    G = c["hq"] // H
    q, seq, pos, table, offs = map(_np, (s.q, s.seq, s.pos, s.table, s.offs))
    codes = s.codes[:, s.layer].cpu().numpy()
    scales = _np(s.scales[:, s.layer])
    sel = np.full((len(seq), H, K), -1, np.int32)
    count = np.zeros((len(seq), H), np.int32)
    for t in np.flatnonzero(seq >= 0):
        n = (offs[seq[t]] + pos[t]) // bs + 1
        blk = table[seq[t], :n]
        for g in range(H):
            x = q[t, g * G:(g + 1) * G]
            unit = np.exp2(_exact_exponent(np.abs(x).max(-1)).astype(np.float64))[:, None]
            x = np.clip(np.rint(x / unit), -127, 127)
            hi, lo = codes[blk, g, 0].astype(np.float64) - 128, codes[blk, g, 1].astype(np.float64) - 128
            score = ((np.maximum(x, 0) @ hi.T + np.minimum(x, 0) @ lo.T) * unit).max(0) * scales[blk, g]
            score[:c["sink"]] = np.inf
            score[max(0, n - c["recent"]):] = np.inf
            best = np.sort(np.argsort(-score, kind="stable")[:K])
            sel[t, g, :len(best)], count[t, g] = best, len(best)
    return {"sel": sel, "count": count}


def _exact_sparse(s, c):
    H, bs = c["hkv"], c["bs"]
    G = c["hq"] // H
    q, seq, pos, table, offs, sel = map(_np, (s.q, s.seq, s.pos, s.table, s.offs, s.sel))
    out = np.zeros(q.shape)
    k, v = _exact_rows(s, c, s.k), _exact_rows(s, c, s.v)
    for t in np.flatnonzero(seq >= 0):
        for g in range(H):
            j = sel[t, g][sel[t, g] >= 0]
            p = (j[:, None] * bs + np.arange(bs)).reshape(-1)
            p = p[(p >= offs[seq[t]]) & (p <= offs[seq[t]] + pos[t])]
            at = (table[seq[t], p // bs], p % bs, g)
            if p.size:
                x = q[t, g * G:(g + 1) * G] @ k[at].T * s.scale
                w = np.exp(x - x.max(-1, keepdims=True))
                out[t, g * G:(g + 1) * G] = w @ v[at] / w.sum(-1, keepdims=True)
    return out
