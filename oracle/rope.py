"""Oracle for rotary positions: a plain CPU restatement in 64 bits.

TEST INFRASTRUCTURE ONLY, like the rest of ``oracle/``; it imports nothing
from the CUDA library.

The pages leave positions to the model that calls the cache; the definition is
the usual one.  Pair ``i`` of a head turns by ``pos * f_i`` with
``f_i = base ** (-2 i / rotary_dim)``: ``(a, b) -> (a c - b s, b c + a s)``,
``c`` and ``s`` the cosine and sine times ``attn_scale``.  Pairs are
``(i, i + rotary_dim / 2)`` or, interleaved, ``(2 i, 2 i + 1)``; the dims from
``rotary_dim`` on pass unchanged.
"""

from __future__ import annotations

import math

import numpy as np

__all__ = ["inv_freq", "attn_factor", "rotate"]


def inv_freq(rotary_dim: int, base: float, scaling=None, factor: float = 1.0,
             original_len: float = 0.0, turns_fast: float = 32.0,
             turns_slow: float = 1.0) -> np.ndarray:
    """Frequencies in radians per token, pair by pair."""
    if scaling == "base":
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    out = []
    for i in range(rotary_dim // 2):
        f = base ** (-2.0 * i / rotary_dim)
        if scaling == "linear":
            f = f / factor
        elif scaling == "by_parts":
            turns = original_len * f / (2 * math.pi)
            if turns >= turns_fast:
                pass
            elif turns <= turns_slow:
                f = f / factor
            else:
                keep = (turns - turns_slow) / (turns_fast - turns_slow)
                f = keep * f + (1 - keep) * f / factor
        out.append(f)
    return np.array(out, dtype=np.float64)


def attn_factor(scaling, factor: float) -> float:
    return 0.1 * math.log(factor) + 1.0 if scaling == "by_parts" else 1.0


def rotate(x: np.ndarray, pos: np.ndarray, freq: np.ndarray, interleaved: bool,
           attn_scale: float = 1.0) -> np.ndarray:
    """Turned ``x`` ([T, H, D], any real type) at positions ``pos`` ([T])."""
    x = np.asarray(x, dtype=np.float64)
    y = x.copy()
    n = len(freq)
    for i in range(n):
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        # the angle modulo one turn in long arithmetic where that is wider
        ang = np.asarray(pos, dtype=np.longdouble) * np.longdouble(freq[i])
        c = (attn_scale * np.cos(ang)).astype(np.float64)[:, None]
        s = (attn_scale * np.sin(ang)).astype(np.float64)[:, None]
        a, b = x[:, :, ia], x[:, :, ib]
        y[:, :, ia] = a * c - b * s
        y[:, :, ib] = b * c + a * s
    return y
