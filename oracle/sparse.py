"""Oracle for sparse decode: key bounds of blocks, block scores and selection,
attention over selected blocks.  A plain, slow CPU restatement in 64 bits.

TEST INFRASTRUCTURE ONLY, like the rest of ``oracle/``; it imports nothing
from the CUDA library.

"mini-runtime ch.12 Paged KV Cache" §6 names sparse KV as a next step of paged
caches and gives no scheme.  The readings taken here:

* A block is described by the extremes ``hi_d`` and ``lo_d`` of its keys, element
  by element: ``q . k <= sum_d max(q_d hi_d, q_d lo_d)`` for each of them.
* The extremes are stored in 8 bits with one power of two per (block, head),
  rounded outwards, and queries are coded the same way (to nearest), so a
  score is a whole number times a power of two and has one value whatever the
  order of its sum: the selection, ties included, is a matter of integers.
* Rows from 0 to the last one a sequence holds count, so that all holders of a
  shared block agree about it.
"""

from __future__ import annotations

import math

import numpy as np

__all__ = ["exponent", "block_bounds", "query_codes", "block_scores", "select",
           "sparse_attention"]

E_MIN, E_MAX = -40, 40


def exponent(absmax: float) -> int:
    """The smallest e in [E_MIN, E_MAX] with absmax <= 127 * 2**e (E_MAX where
    there is none)."""
    if math.isnan(absmax):
        return E_MAX
    e = E_MIN
    while e < E_MAX and absmax > math.ldexp(127.0, e):
        e += 1
    return e


def _clip(x: float, nan: int, f) -> int:
    if math.isnan(x):
        return nan
    if math.isinf(x):
        return 127 if x > 0 else -127
    return max(-127, min(127, int(f(x))))


def block_bounds(rows: np.ndarray):
    """Key rows ``[n, D]`` of one block and head -> codes int ``[2, D]`` (hi,
    lo) and the exponent."""
    rows = np.asarray(rows, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        hi, lo = rows.max(0), rows.min(0)      # NaN propagates
    e = exponent(float(np.max(np.maximum(np.abs(hi), np.abs(lo)))))
    unit = math.ldexp(1.0, e)
    return np.array([[_clip(x / unit, 127, math.ceil) for x in hi],
                     [_clip(x / unit, -127, math.floor) for x in lo]]), e


def query_codes(q: np.ndarray):
    """One head's query ``[D]`` -> codes int ``[D]`` and the exponent."""
    q = np.asarray(q, dtype=np.float64)
    e = exponent(float(np.max(np.abs(q))))
    unit = math.ldexp(1.0, e)
    return np.array([_clip(x / unit, 0, lambda y: round(y)) for x in q]), e


def block_scores(q: np.ndarray, codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """Queries ``[G, D]`` of one kv head, codes ``[n, 2, D]``, scales ``[n]`` ->
    scores ``[n]``."""
    best = np.full(len(codes), -np.inf)
    for x in q:
        c, e = query_codes(x)
        dot = np.where(c >= 0, c * codes[:, 0].astype(np.int64), c * codes[:, 1].astype(np.int64))
        best = np.maximum(best, dot.sum(-1).astype(np.float64) * math.ldexp(1.0, e))
    return best * np.asarray(scales, dtype=np.float64)


def select(scores: np.ndarray, k: int, sink: int, recent: int) -> list:
    """The selected entries, ascending."""
    n = len(scores)
    if n <= k:
        return list(range(n))
    taken = list(range(sink)) + list(range(n - recent, n))
    rest = sorted(range(sink, n - recent), key=lambda j: (-scores[j], j))
    return sorted(taken + rest[:k - len(taken)])


def sparse_attention(q: np.ndarray, keys: np.ndarray, values: np.ndarray, entries, block_size: int,
                     offset: int, pos: int, scale: float):
    """Queries ``[G, D]`` of one kv head over the listed table entries of a
    sequence whose table rows are ``keys``, ``values`` ``[blocks, bs, D]`` (by
    table entry).  Returns ``out [G, D]``, the weighted mean of |V| and the
    largest sum of |q| |k| (for error bounds)."""
    at = [(j, r) for j in entries if j >= 0 for r in range(block_size)
          if offset <= j * block_size + r <= offset + pos]
    G, D = q.shape
    if not at:
        return np.zeros((G, D)), np.zeros((G, D)), np.zeros(G)
    j, r = np.array(at).T
    K, V = keys[j, r].astype(np.float64), values[j, r].astype(np.float64)
    s = q.astype(np.float64) @ K.T * scale
    w = np.exp(s - s.max(-1, keepdims=True))
    w /= w.sum(-1, keepdims=True)
    return w @ V, w @ np.abs(V), (np.abs(q.astype(np.float64)) @ np.abs(K).T).max(-1)
