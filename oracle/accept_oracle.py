"""Oracle of the acceptance of drafted tokens: plain numpy, fp64, one request at a time.

The walk of the rejection rule in its recursive form: at a node the target's distribution is replaced, after each
rejected child, by the normalised residual max(p - q, 0), q the distribution that child was drawn from (a point mass
where the draft chose it).  Imported by the tests only; shares no code with the CUDA library.
"""
from __future__ import annotations

from typing import Optional, Sequence

import numpy as np


def softmax(z: np.ndarray) -> np.ndarray:
    e = np.exp(z - z.max())
    return e / e.sum()


def residual(p: np.ndarray, q: np.ndarray) -> np.ndarray:
    """Distribution left after a rejection; p itself where nothing is left."""
    r = np.maximum(p - q, 0.0)
    return r / r.sum() if r.sum() > 0 else p


def accept(parent: Sequence[int], tokens: Sequence[int], logits: np.ndarray, uniform: Optional[np.ndarray],
           gumbel: Optional[np.ndarray], temperature: float, draft: Optional[np.ndarray] = None):
    """-> (path, next token).  logits, draft [n, V]; uniform [n]; gumbel [V]."""
    n, V = len(parent), logits.shape[1]
    node, path = 0, []
    while True:
        path.append(node)
        z = logits[node].astype(np.float64)
        if np.isnan(z).any() or not np.isfinite(z.max()):
            return path, -1
        kids = [j for j in range(n) if parent[j] == node]
        took = -1
        if temperature == 0:
            best = int(np.argmax(z))
            for j in kids:
                if tokens[j] == best:
                    took = j
                    break
        else:
            p = softmax(z / temperature)
            for j in kids:
                t = tokens[j]
                q = np.zeros(V)
                if draft is not None:
                    q = draft[node].astype(np.float64)
                elif 0 <= t < V:
                    q[t] = 1.0
                if 0 <= t < V and uniform[j] * q[t] < p[t]:
                    took = j
                    break
                p = residual(p, q)
        if took < 0:
            if temperature == 0:
                return path, best
            with np.errstate(divide="ignore"):
                return path, int(np.argmax(np.log(p) + gumbel.astype(np.float64)))
        node = took
