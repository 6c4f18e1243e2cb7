"""Timed cases of windowed attention and of tree verification over the paged cache.

Four operators:

``window``   decode attention with a sliding window and a few first tokens that
             stay visible (``pkv.decode_attention_window``);
``prefill``  the same for the new tokens of prompts and chunks
             (``pkv.prefill_attention_window``);
``tree``     attention of drafted tokens over their context and, by a mask, over
             one another (``pkv.decode_attention_tree``);
``accept``   the rows of the accepted drafted tokens moved right behind the
             context (``pkv.accept_tokens``).

With ``own`` false ``run`` computes them with elementary torch operations, with
``own`` true through the library.  ``exact`` is the definition in 64 bits.
"""

import math
import zlib
from types import SimpleNamespace

import numpy as np
import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32, "i8": torch.bfloat16}  # of q and out


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one user decoding at the end of a long context, a window of 4096: latency
        dict(name="window_one_131072", op="window", dtype="bf16", hq=32, hkv=8, d=128, bs=16, layers=1,
             seqs=1, len_lo=131072, len_hi=131072, window=4096, sink=4, offsets=False),
        # an ordinary decode batch, some sequences shorter than the window
        dict(name="window_batch_64", op="window", dtype="bf16", hq=32, hkv=8, d=128, bs=16, layers=1,
             seqs=64, len_lo=512, len_hi=8192, window=2048, sink=4, offsets=True),
        # the same from an int8 pool
        dict(name="window_batch_64_i8", op="window", dtype="i8", hq=32, hkv=8, d=128, bs=16, layers=1,
             seqs=64, len_lo=512, len_hi=8192, window=2048, sink=4, offsets=True),
        # prompts of a model with window layers
        dict(name="prefill_prompts", op="prefill", dtype="bf16", hq=32, hkv=8, d=128, bs=16, layers=1,
             seqs=8, new_lo=1024, new_hi=8192, ctx_lo=0, ctx_hi=0, window=1024, sink=4, offsets=True),
        # chunks of long prompts after a cached context, 8 query heads a kv head, no first tokens
        dict(name="prefill_chunks", op="prefill", dtype="bf16", hq=64, hkv=8, d=128, bs=16, layers=1,
             seqs=4, new_lo=500, new_hi=1000, ctx_lo=8192, ctx_hi=32768, window=4096, sink=0, offsets=False),
        # fp32, head_dim 64, three query heads a kv head, a window of 100 tokens
        dict(name="prefill_f32", op="prefill", dtype="f32", hq=12, hkv=4, d=64, bs=32, layers=2,
             seqs=5, new_lo=1, new_hi=700, ctx_lo=0, ctx_hi=300, window=100, sink=1, offsets=True),
        # one user, 24 drafted tokens: latency
        dict(name="tree_one_16384", op="tree", dtype="bf16", hq=32, hkv=8, d=128, bs=16, layers=1,
             seqs=1, new_lo=24, new_hi=24, ctx_lo=16384, ctx_hi=16384, window=0, sink=0, offsets=False),
        # a batch, the widest trees of one mask word
        dict(name="tree_batch_16", op="tree", dtype="bf16", hq=32, hkv=8, d=128, bs=16, layers=1,
             seqs=16, new_lo=64, new_hi=64, ctx_lo=1024, ctx_hi=16384, window=0, sink=0, offsets=True),
        # a larger batch with small trees, int8 pool
        dict(name="tree_batch_32_i8", op="tree", dtype="i8", hq=32, hkv=8, d=128, bs=16, layers=1,
             seqs=32, new_lo=4, new_hi=8, ctx_lo=1024, ctx_hi=8192, window=0, sink=0, offsets=True),
        # fp32, head_dim 64, a window layer
        dict(name="tree_window_f32", op="tree", dtype="f32", hq=20, hkv=4, d=64, bs=16, layers=2,
             seqs=9, new_lo=3, new_hi=17, ctx_lo=1, ctx_hi=3000, window=512, sink=4, offsets=True),
        # after one user's verification, all 32 layers
        dict(name="accept_one", op="accept", dtype="bf16", hkv=8, d=128, bs=16, layers=32,
             seqs=1, new_lo=24, new_hi=24, ctx_lo=200, ctx_hi=200, accept=5, offsets=False),
        # a batch
        dict(name="accept_batch_64", op="accept", dtype="bf16", hkv=8, d=128, bs=16, layers=16,
             seqs=64, new_lo=32, new_hi=64, ctx_lo=1, ctx_hi=64, accept=8, offsets=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


# products of a drawn case at most: the largest listed cases of bf16 and, with fewer, of the others
_MOST = {"bf16": 300 * 10 ** 9, "i8": 60 * 10 ** 9, "f32": 25 * 10 ** 9}


def draw(rng):
    op = rng.choice(["window", "prefill", "tree", "accept"])
    dtype = rng.choice(["bf16", "bf16", "i8", "f32"])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 4, 5, 8, 16])
    c = dict(op=op, dtype=dtype, hkv=hkv, d=d, bs=rng.choice([8, 16, 16, 32, 64]), layers=rng.choice([1, 2]),
             offsets=rng.random() < 0.5)
    if op == "window":
        hi = _log(rng, 20, 32768)
        c.update(hq=hq, seqs=max(1, min(_log(rng, 1, 64), 400000 // hi)), len_lo=max(1, hi // 16), len_hi=hi,
                 window=_log(rng, 1, 8192), sink=rng.choice([0, 1, 4, 64]))
    elif op == "prefill":
        window, hi, ctx = _log(rng, 1, 4096), _log(rng, 1, 4096), rng.choice([0, 100, 5000, 20000])
        most = _MOST[dtype] // (4 * d * hq)
        while hi * min(window + 64, hi + ctx) > most:
            hi = hi // 2 + 1
        c.update(hq=hq, seqs=max(1, min(_log(rng, 1, 16), most // (hi * min(window + 64, hi + ctx)))),
                 new_lo=max(1, hi // 8), new_hi=hi, ctx_lo=0, ctx_hi=ctx, window=window, sink=rng.choice([0, 1, 4, 64]))
    elif op == "tree":
        n, hi = _log(rng, 1, 128), _log(rng, 1, 32768)
        most = _MOST[dtype] // (4 * d * hq)
        while n * (hi + n) > most:
            n = n // 2 + 1
        c.update(hq=hq, seqs=max(1, min(_log(rng, 1, 32), 260000 // hi, most // (n * (hi + n)))),
                 new_lo=max(1, n // 2), new_hi=n, ctx_lo=hi // 8, ctx_hi=hi,
                 window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]), sink=rng.choice([0, 4]))
    else:
        n = _log(rng, 2, 128)
        c.update(seqs=_log(rng, 1, 64), layers=_log(rng, 1, 16), new_lo=max(1, n // 2), new_hi=n, ctx_lo=1, ctx_hi=40,
                 accept=_log(rng, 1, n))
    return c


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _row_bytes(c):
    return c["hkv"] * c["d"] + (4 * c["hkv"] + 15) // 16 * 16


def _new_pool(c, n, gen):
    """K or V cache of ``n`` blocks: N(0, 1) rows, or int8 codes and scales of such rows."""
    H, D = c["hkv"], c["d"]
    if c["dtype"] != "i8":
        return torch.randn((n, c["layers"], c["bs"], H, D), generator=gen, device="cuda", dtype=DTYPE[c["dtype"]])
    p = torch.zeros((n, c["layers"], c["bs"], _row_bytes(c)), dtype=torch.uint8, device="cuda")
    codes = (torch.randn(p.shape[:3] + (H * D,), generator=gen, device="cuda") * 42).round_().clamp_(-127, 127)
    p[..., :H * D] = (codes + 128).to(torch.uint8)
    scales = torch.rand(p.shape[:3] + (H,), generator=gen, device="cuda") * 0.03 + 0.01
    p[..., H * D:H * D + 4 * H] = scales.view(torch.uint8).view(p.shape[:3] + (4 * H,))
    return p


def _cuda(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dtype)


def _shapes(c):
    """New tokens, lengths, offsets and trees of a case are the same multiset for every seed, so that a case has one
    size of cache and one amount of work; a seed gives their order."""
    f = np.random.RandomState(zlib.crc32(repr(sorted((k, v) for k, v in c.items() if k != "name")).encode()))
    B = c["seqs"]
    if c["op"] == "window":
        new, lens = np.ones(B, np.int64), f.randint(c["len_lo"], c["len_hi"] + 1, B)
    else:
        new = f.randint(c["new_lo"], c["new_hi"] + 1, B)
        lens = new + f.randint(c["ctx_lo"], c["ctx_hi"] + 1, B)
    offs = f.randint(0, c["bs"], B) if c["offsets"] else np.zeros(B, np.int64)
    # a drafted token hangs on one of the eight before it, or on the context
    trees = [[f.randint(-1, i) if i < 8 else f.randint(i - 8, i) for i in range(n)] for n in new] \
        if c["op"] == "tree" else [None] * B
    # accepted tokens, and how many of them stay where they are
    count = np.minimum(f.randint(0, c["accept"] + 1, B) if B > 1 else c["accept"], new) if c["op"] == "accept" else new
    stay = np.array([f.randint(max(0, 2 * k - n), k + 1) for k, n in zip(count, new)]) if B > 1 \
        else np.maximum(0, 2 * count - new)
    return new, lens, offs, trees, count, stay


def _ancestors(tree):
    """[n, n] truth values (token i sees token j: itself and what it hangs on) and the depths of a tree."""
    n = len(tree)
    sees, depth = np.zeros((n, n), bool), np.zeros(n, np.int64)
    for i, parent in enumerate(tree):
        if parent >= 0:
            sees[i] = sees[parent]
            depth[i] = depth[parent] + 1
        sees[i, i] = True
    return sees, depth


def prepare(case, seed):
    c = case
    r = np.random.RandomState(seed % (1 << 31))
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = SimpleNamespace(case=c, op=c["op"], layer=c["layers"] - 1, scale=c["d"] ** -0.5)
    new, lens, offs, trees, count, stay = _shapes(c)
    order = r.permutation(c["seqs"])
    new, lens, offs, count, stay = (x[order] for x in (new, lens, offs, count, stay))
    trees = [trees[i] for i in order]
    nblk = -(-(offs + lens) // c["bs"])
    n = int(nblk.sum())
    ids, table, at = r.permutation(n), np.full((c["seqs"], int(nblk.max())), -1, np.int64), 0
    for b in range(c["seqs"]):
        table[b, :nblk[b]] = ids[at:at + nblk[b]]
        at += nblk[b]
    s.new, s.cu = new, np.concatenate([[0], np.cumsum(new)])  # also known on the host
    s.lens, s.offs, s.table, s.cu_q = _cuda(lens), _cuda(offs), _cuda(table), _cuda(s.cu, torch.int64)
    s.host_lens = lens
    s.k, s.v = _new_pool(c, n, gen), _new_pool(c, n, gen)
    if own:
        import paged_kv_cache_blk_gb300 as pkv
        s.pkv = pkv
        s.pool = pkv.Pool(s.k, s.v, c["hkv"], c["d"]) if c["dtype"] == "i8" else pkv.Pool(s.k, s.v)
    if c["op"] == "accept":
        # a path keeps its first tokens in place and goes on behind the accepted ones: a pass can be repeated
        path = np.full((c["seqs"], c["accept"]), -1, np.int64)
        for b, (n, k, j) in enumerate(zip(new, count, stay)):
            path[b, :k] = np.concatenate([np.arange(j), np.sort(r.choice(np.arange(k, n), k - j, replace=False))])
        s.path, s.count = _cuda(path), _cuda(count)
        return s
    s.q = torch.randn((int(s.cu[-1]), c["hq"], c["d"]), generator=gen, device="cuda", dtype=DTYPE[c["dtype"]])
    s.out = torch.zeros_like(s.q)
    if c["op"] == "tree":
        words = -(-c["new_hi"] // 64)
        mask, q_pos = np.zeros((len(s.q), words), np.uint64), np.zeros(len(s.q), np.int64)
        for b, tree in enumerate(trees):
            sees, depth = _ancestors(tree)
            q_pos[s.cu[b]:s.cu[b + 1]] = lens[b] - new[b] + depth
            bits = np.zeros((len(tree), words * 64), np.uint8)
            bits[:, :len(tree)] = sees
            mask[s.cu[b]:s.cu[b + 1]] = np.packbits(bits, axis=1, bitorder="little").view(np.uint64)
        s.mask, s.q_pos = _cuda(mask.view(np.int64), torch.int64), _cuda(q_pos)
        if own:
            s.workspace = torch.empty(s.pkv.decode_tree_workspace_size(s.pool, c["seqs"], c["hq"], c["new_hi"]),
                                      dtype=torch.uint8, device="cuda")
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(state):
    s = state
    if own:
        return _OWN[s.op](s)
    return _PLAIN[s.op](s)


def _own_window(s):
    c = s.case
    s.pkv.decode_attention_window(s.pool, s.layer, s.q, s.scale, s.table, s.lens, s.offs, c["window"], s.out,
                                  sink=c["sink"])
    return s.out


def _own_prefill(s):
    c = s.case
    s.pkv.prefill_attention_window(s.pool, s.layer, s.q, s.scale, s.table, s.lens, s.offs, s.cu_q, c["new_hi"],
                                   c["window"], s.out, sink=c["sink"])
    return s.out


def _own_tree(s):
    c = s.case
    s.pkv.decode_attention_tree(s.pool, s.layer, s.q, s.scale, s.table, s.lens, s.offs, s.cu_q, c["new_hi"], s.mask,
                                s.out, s.workspace, q_pos=s.q_pos, window=c["window"], sink=c["sink"])
    return s.out


def _own_accept(s):
    s.pkv.accept_tokens(s.pool, -1, s.table, s.lens, s.offs, s.cu_q, s.path, s.count)
    return {"k": _values(s, s.k), "v": _values(s, s.v)}


def _values(s, cache):
    """What a cache holds: itself, or the numbers that int8 codes and scales stand for, in the type of the rows."""
    c = s.case
    if c["dtype"] != "i8":
        return cache
    HD, H = c["hkv"] * c["d"], c["hkv"]
    codes = (cache[..., :HD] - 128.0).unflatten(-1, (H, c["d"]))
    scales = cache[..., HD:HD + 4 * H].view(torch.float32)[..., None]
    return torch.mul(codes, scales, out=torch.empty(codes.shape, dtype=DTYPE["i8"], device="cuda"))


def _rows(s, cache, blk, row):
    """Rows of the layer, all heads, in 32 bits."""
    c = s.case
    x = cache[blk, s.layer, row]
    if c["dtype"] != "i8":
        return x.float()
    HD, H = c["hkv"] * c["d"], c["hkv"]
    codes = (x[..., :HD] - 128.0).unflatten(-1, (H, c["d"]))
    return codes.mul_(x[..., HD:HD + 4 * H].contiguous().view(torch.float32)[..., None])


def _softmax_v(x, seen, v):
    """Weights of the scores that are seen, times v; zeros where nothing is."""
    x = torch.where(seen, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    w = (x - torch.where(top > -math.inf, top, 0.0)).exp_()
    total = w.sum(-1, keepdim=True)
    return (w @ v) / torch.where(total > 0, total, 1.0)


def _plain_window(s):
    c = s.case
    W, S, bs = c["window"], c["sink"], c["bs"]
    W = min(W, s.table.shape[1] * bs)
    lens = s.lens.long()[:, None]
    first = (lens - W).clamp(min=0)
    sink = torch.arange(S, device="cuda").expand(c["seqs"], S)
    window = first + torch.arange(W, device="cuda")
    pos = torch.cat([sink, window], 1)
    seen = torch.cat([sink < first, window < lens], 1)
    p = torch.where(seen, pos, 0) + s.offs.long()[:, None]
    blk, row = s.table.gather(1, p // bs).long(), p % bs
    k = _rows(s, s.k, blk, row).permute(0, 2, 3, 1)  # [B, H, D, keys]
    x = (s.q.float().unflatten(1, (c["hkv"], -1)) @ k) * s.scale
    del k
    v = _rows(s, s.v, blk, row).transpose(1, 2)
    return _softmax_v(x, seen[:, None, None], v).flatten(1, 2).to(s.q.dtype)


def _sequence(s, b, lo, hi):
    """K [H, D, keys] and V [H, keys, D] of positions lo .. hi - 1 of a sequence."""
    p = torch.arange(lo, hi, device="cuda") + s.offs[b].long()
    blk, row = s.table[b, p // s.case["bs"]].long(), p % s.case["bs"]
    return _rows(s, s.k, blk, row).permute(1, 2, 0), _rows(s, s.v, blk, row).transpose(0, 1)


def _plain_prefill(s):
    c = s.case
    W, S, H = c["window"], c["sink"], c["hkv"]
    out = torch.empty_like(s.q)
    for b in range(c["seqs"]):
        n, ctx = int(s.new[b]), int(s.host_lens[b] - s.new[b])
        low = max(0, ctx - W + 1)
        k0, v0 = _sequence(s, b, 0, min(S, low))
        k1, v1 = _sequence(s, b, low, ctx + n)
        for i in range(0, n, 512):
            m = min(512, n - i)
            lo, hi = max(low, ctx + i - W + 1), ctx + i + m
            some = min(S, lo)  # first tokens that are not among lo .. hi - 1
            k = torch.cat([k0, k1[:, :, :max(0, some - low)], k1[:, :, lo - low:hi - low]], 2)
            v = torch.cat([v0, v1[:, :max(0, some - low)], v1[:, lo - low:hi - low]], 1)
            key = torch.cat([torch.arange(some, device="cuda"), torch.arange(lo, hi, device="cuda")])
            pos = torch.arange(ctx + i, hi, device="cuda")[:, None]
            seen = (key <= pos) & ((key > pos - W) | (key < S))
            at = s.cu[b] + i
            q = s.q[at:at + m].float().unflatten(1, (H, -1)).permute(1, 2, 0, 3)  # [H, G, m, D]
            x = (q.flatten(1, 2) @ k).mul_(s.scale)
            o = _softmax_v(x.unflatten(1, (-1, m)), seen, v[:, None]).permute(2, 0, 1, 3)
            out[at:at + m] = o.flatten(1, 2).to(out.dtype)
    return out


def _plain_tree(s):
    c = s.case
    W, S, H = c["window"], c["sink"], c["hkv"]
    out = torch.empty_like(s.q)
    for b in range(c["seqs"]):
        n, ctx, at = int(s.new[b]), int(s.host_lens[b] - s.new[b]), int(s.cu[b])
        k, v = _sequence(s, b, 0, ctx + n)
        bits = (s.mask[at:at + n, :, None] >> torch.arange(64, device="cuda")) & 1
        key = torch.arange(ctx, device="cuda")
        old = torch.ones((n, ctx), dtype=torch.bool, device="cuda")
        if W:
            old = (key > s.q_pos[at:at + n, None] - W) | (key < S)
        seen = torch.cat([old, bits.flatten(1)[:, :n] == 1], 1)
        q = s.q[at:at + n].float().unflatten(1, (H, -1)).permute(1, 2, 0, 3)
        x = (q.flatten(1, 2) @ k).mul_(s.scale)
        o = _softmax_v(x.unflatten(1, (-1, n)), seen, v[:, None]).permute(2, 0, 1, 3)
        out[at:at + n] = o.flatten(1, 2).to(out.dtype)
    return out


def _plain_accept(s):
    bs, M = s.case["bs"], s.path.shape[1]
    k = torch.arange(M, device="cuda")
    first = (s.offs + s.lens).long() - (s.cu_q[1:] - s.cu_q[:-1])  # table position of the first drafted token
    # entries behind the accepted ones move the first drafted token onto itself or to where the path puts it
    live = k < s.count[:, None]
    src = first[:, None] + torch.where(live, s.path, torch.where(s.count[:, None] > 0, s.path[:, :1], 0)).long()
    dst = first[:, None] + torch.where(live, k, 0)
    sb, db = s.table.gather(1, src // bs).long(), s.table.gather(1, dst // bs).long()
    for cache in (s.k, s.v):
        cache[db, :, dst % bs] = cache[sb, :, src % bs]
    return {"k": _values(s, s.k), "v": _values(s, s.v)}


_OWN = {"window": _own_window, "prefill": _own_prefill, "tree": _own_tree, "accept": _own_accept}
_PLAIN = {"window": _plain_window, "prefill": _plain_prefill, "tree": _plain_tree, "accept": _plain_accept}


# --------------------------------------------------------------------------
# the work of one pass
# --------------------------------------------------------------------------

def work(case):
    c = case
    H, D = c["hkv"], c["d"]
    io = 4 if c["dtype"] == "f32" else 2
    row = {"bf16": 2, "f32": 4, "i8": 1}[c["dtype"]] * D + (4 if c["dtype"] == "i8" else 0)  # one head of a token
    new, lens, offs, trees, count, stay = _shapes(c)
    ctx = lens - new
    if c["op"] == "accept":
        return {"bytes": max(1, int((count - stay).sum())) * c["layers"] * 2 * 2 * H * row, "flops": 0}
    W = c["window"] or int(lens.max())
    S = c["sink"]
    low = np.maximum(0, ctx - W + 1)  # the first key of the first window
    keys = int((lens - low + np.minimum(S, low)).sum())
    pairs = 0
    for b in range(c["seqs"]):
        if c["op"] == "tree":
            sees, depth = _ancestors(trees[b])
            first = np.maximum(0, ctx[b] + depth - W + 1)
            old = np.maximum(0, ctx[b] - first) + np.minimum(S, np.minimum(first, ctx[b]))
            pairs += int(sees.sum() + old.sum())
        else:
            pos = ctx[b] + np.arange(new[b])
            first = np.maximum(0, pos - W + 1)
            pairs += int((pos + 1 - first + np.minimum(S, first)).sum())
    q = int(new.sum()) * c["hq"]
    extra = int(new.sum()) * (-(-c["new_hi"] // 64) * 8 + 4) if c["op"] == "tree" else 0
    return {"bytes": keys * H * 2 * row + q * 2 * D * io + extra, "flops": pairs * c["hq"] * D * 4}


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_accept(s, case) if case["op"] == "accept" else _exact_attention(s, case)


def _exact_rows(s, c, cache, b, keys):
    """[H, keys, D] of listed positions of a sequence."""
    at = keys + int(s.offs[b])
    a = cache[s.table[b][at // c["bs"]].long(), s.layer, at % c["bs"]]
    H, D = c["hkv"], c["d"]
    if c["dtype"] == "i8":
        unit = a[:, H * D:H * D + 4 * H].contiguous().view(torch.float32).double()
        a = (a[:, :H * D].double() - 128).view(-1, H, D) * unit[:, :, None]
    return a.double().transpose(0, 1)


def _exact_attention(s, c):
    G = c["hq"] // c["hkv"]
    W, S = c["window"], c["sink"]
    out = torch.zeros(s.q.shape, dtype=torch.float64, device="cuda")
    for b in range(c["seqs"]):
        n, ctx = int(s.new[b]), int(s.host_lens[b] - s.new[b])
        for i0 in range(0, n, 256):
            i1 = min(n, i0 + 256)
            low = max(0, ctx + i0 - W + 1) if W and c["op"] != "tree" else max(0, ctx - W + 1) if W else 0
            top = ctx + n if c["op"] == "tree" else ctx + i1
            keys = torch.tensor([j for j in range(min(S, low))] + [j for j in range(low, top)], device="cuda")
            hide = torch.zeros((i1 - i0, len(keys)), dtype=torch.bool, device="cuda")
            for i in range(i0, i1):
                t = int(s.cu[b]) + i
                if c["op"] == "tree":
                    if W:
                        hide[i - i0] = (keys <= int(s.q_pos[t]) - W) & (keys >= S) & (keys < ctx)
                    word = [int(w) for w in s.mask[t]]
                    drafted = [not word[j // 64] >> (j % 64) & 1 for j in range(n)]
                    hide[i - i0, len(keys) - n:] = torch.tensor(drafted, device="cuda")
                else:
                    pos = ctx + i
                    hide[i - i0] = (keys > pos) | ((keys <= pos - W) & (keys >= S))
            k, v = (_exact_rows(s, c, x, b, keys) for x in (s.k, s.v))
            rows = slice(int(s.cu[b]) + i0, int(s.cu[b]) + i1)
            for h in range(c["hq"]):
                x = s.q[rows, h].double() @ k[h // G].T * s.scale
                x[hide] = -math.inf
                w = torch.softmax(x, -1)
                out[rows, h] = torch.where(hide.all(-1)[:, None], 0.0, w @ v[h // G])
    return out


def _exact_accept(s, c):
    offs, table, path, count = (x.cpu().numpy() for x in (s.offs, s.table, s.path, s.count))
    got = {}
    for name in ("k", "v"):
        cache = _values(s, getattr(s, name)).double()
        old = cache.clone()
        for b in range(c["seqs"]):
            first = int(offs[b] + s.host_lens[b] - s.new[b])
            for j in range(int(count[b])):
                src, dst = first + int(path[b, j]), first + j
                cache[table[b, dst // c["bs"]], :, dst % c["bs"]] = old[table[b, src // c["bs"]], :, src % c["bs"]]
        got[name] = cache
    return got
