"""Oracle of the 4-bit key/value cache and the attention over it: plain numpy, fp64, token by token.

States the format (one group at a time, from its words), and softmax attention as its definition: one row at a time
over the list of tokens the row sees.  Imported by the tests only; shares no code with the CUDA library.
"""
from __future__ import annotations

from typing import List, Optional, Sequence, Tuple

import numpy as np

PAGE = 64
GROUP = 32


def round_bf16(x: float) -> float:
    """Nearest value with 8 significant bits (ties to even), as bf16 has in its normal range."""
    if x == 0 or not np.isfinite(x):
        return x
    m, e = np.frexp(x)
    return float(np.ldexp(np.rint(m * 256.0), e - 8))


def quantise_group(x: np.ndarray) -> Tuple[np.ndarray, float]:
    """One group of 32 values -> (codes -8..7, scale)."""
    x = np.asarray(x, dtype=np.float64)
    if not np.all(np.isfinite(x)):
        return np.zeros(GROUP, dtype=np.int64), float("nan")
    m = x[int(np.argmax(np.abs(x)))]         # argmax: the first of equals
    d = round_bf16(-m / 8.0)
    d = float(np.float16(min(max(d, -2720.0), 2720.0)))
    if d == 0:
        return np.zeros(GROUP, dtype=np.int64), d
    return np.clip(np.rint(x / d), -8, 7).astype(np.int64), d


def quantise_row(x: np.ndarray) -> np.ndarray:
    """Values a row of D channels stands for in the cache."""
    out = np.empty(len(x))
    for g in range(0, len(x), GROUP):
        c, d = quantise_group(x[g:g + GROUP])
        out[g:g + GROUP] = c * d
    return out


def nibble(e: int) -> int:
    return (e >> 1) + 4 * (e & 1)


def block_rows(block: np.ndarray, D: int) -> Tuple[np.ndarray, np.ndarray]:
    """One 72 D-byte block -> keys [64, D] and values [64, D], bit by bit as the format is written down."""
    raw = np.ascontiguousarray(block, dtype=np.uint8)
    words = raw.view("<u4")
    halves = raw.view("<f2").astype(np.float64)
    k, v = np.empty((PAGE, D)), np.empty((PAGE, D))
    for r in range(PAGE):
        x = {256: ((r & 1) << 2) | ((r >> 1) & 3), 128: (r >> 1) & 3, 64: (r >> 2) & 1}[D]
        for c in range(D):
            w = int(words[r * (D // 8) + (((c // 32) ^ x) * 4) + (c % 32) // 8])
            k[r, c] = (((w >> (4 * nibble(c % 8))) & 15) - 8) * halves[16 * D + r * (D // 32) + c // 32]
            w = int(words[9 * D + ((r // 32 * (D // 4) + c // 4) * 4 + r // 8 % 4) * 4 + c % 4])
            v[r, c] = (((w >> (4 * nibble(r % 8))) & 15) - 8) * halves[34 * D + (c // 32) * PAGE + r]
    return k, v


def root_path(parent: Sequence[int], i: int) -> List[int]:
    path = []
    while i >= 0:
        path.append(i)
        i = int(parent[i])
    return path


def attention_row(q: np.ndarray, keys: np.ndarray, values: np.ndarray, scale: float) -> np.ndarray:
    """softmax(scale q . k) v over the given tokens; zeros where there are none."""
    if len(keys) == 0:
        return np.zeros(values.shape[-1])
    s = scale * (keys @ q)
    w = np.exp(s - s.max())
    return (w / w.sum()) @ values


def tree_attention(q: np.ndarray, keys: np.ndarray, values: np.ndarray, k_new: Optional[np.ndarray],
                   v_new: Optional[np.ndarray], parent: Sequence[int], scale: float) -> np.ndarray:
    """q [n, Hq, D]; keys, values [L, Hkv, D] committed rows; k_new, v_new [n, Hkv, D] or None -> [n, Hq, D]."""
    n, Hq, D = q.shape
    Hkv = keys.shape[1]
    out = np.zeros((n, Hq, D))
    for i in range(n):
        path = root_path(parent, i)
        for h in range(Hq):
            g = h // (Hq // Hkv)
            k, v = keys[:, g], values[:, g]
            if k_new is not None:
                k = np.concatenate([k, k_new[path, g]])
                v = np.concatenate([v, v_new[path, g]])
            out[i, h] = attention_row(q[i, h].astype(np.float64), k.astype(np.float64), v.astype(np.float64), scale)
    return out
