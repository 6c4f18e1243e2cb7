"""Oracle for windowed attention and tree verification: which keys a query sees,
attention over them in 64 bits, and the moves of accepted tokens.  A plain, slow
CPU restatement.

TEST INFRASTRUCTURE ONLY, like the rest of ``oracle/``; it imports nothing
from the CUDA library.

"vLLM PagedAttention source notes" §2.3 computes attention over what the block
table names; the masks are this library's readings:

* A window of W tokens and S first tokens: position P sees the keys ``i <= P``
  with ``i > P - W`` or ``i < S``.
* Drafted tokens behind a context of C tokens: query i sees the context (under
  the window, from its own position along the tree) and the drafted tokens
  whose bit is set in its mask.
* An accepted path ``a_0 < a_1 < ...`` of drafted tokens: the rows of position
  ``C + a_k`` go to position ``C + k``, as if all were read before any is written.
"""

from __future__ import annotations

import numpy as np

__all__ = ["window_seen", "tree_seen", "mask_words", "attention", "accept_moves"]


def window_seen(pos: int, window: int, sink: int) -> np.ndarray:
    """Keys 0..pos that the query at ``pos`` sees (window 0: all)."""
    return np.array([window == 0 or i > pos - window or i < sink for i in range(pos + 1)], bool)


def tree_seen(ctx: int, sees: np.ndarray, i: int, pos: int, window: int, sink: int) -> np.ndarray:
    """Keys 0..ctx + n - 1 that drafted token ``i`` at position ``pos`` sees;
    ``sees`` [n, n]: which drafted tokens each sees."""
    pos = max(pos, ctx)
    old = [window == 0 or k > pos - window or k < sink for k in range(ctx)]
    return np.array(old + [bool(x) for x in sees[i]], bool)


def mask_words(sees: np.ndarray, words: int) -> np.ndarray:
    """[n, n] truth values as uint64 [n, words], bit j of a row in word j // 64."""
    out = np.zeros((len(sees), words), np.uint64)
    for i, row in enumerate(sees):
        for j in np.flatnonzero(row):
            out[i, j // 64] |= np.uint64(1) << np.uint64(j % 64)
    return out


def attention(q: np.ndarray, k: np.ndarray, v: np.ndarray, seen: np.ndarray, scale: float):
    """One kv head: q [G, D], k and v [n, D] in 64 bits, ``seen`` [n] -> the
    result [G, D]; sum of weight times |v|, the size of what is summed
    [G, D]; the largest sum of |q_d k_d| over a seen key [G]."""
    G, D = q.shape
    out, mean, top = np.zeros((G, D)), np.zeros((G, D)), np.zeros(G)
    k, v = k[seen], v[seen]
    for h in range(G):
        if not len(k):
            continue
        s = scale * (k @ q[h])
        if np.all(s == -np.inf):
            continue
        w = np.exp(s - s.max())
        w /= w.sum()
        out[h], mean[h] = w @ v, w @ np.abs(v)
        top[h] = (np.abs(k) @ np.abs(q[h])).max()
    return out, mean, top


def accept_moves(first: int, path) -> list:
    """(source, destination) positions; ``first``: that of the first drafted token."""
    return [(first + int(a), first + k) for k, a in enumerate(path) if int(a) != k]
