"""Plain fp64 statements of sequences through one GDN layer and of log-probabilities of rows of logits.

TEST INFRASTRUCTURE ONLY, like gdn_oracle.py, whose token step this replays.  The chunked form is stated here once more
on its own (``chunk_step``), from the formulas the kernels use, and pinned to the replay by the tests.
"""
from __future__ import annotations

import math
from typing import List, Optional, Sequence, Tuple

import numpy as np

from . import gdn_oracle as O


def run_sequence(T: np.ndarray, W: np.ndarray, x: np.ndarray, beta: np.ndarray, log_g: np.ndarray,
                 conv_w: Optional[np.ndarray], d: O.Dims) -> Tuple[np.ndarray, np.ndarray, np.ndarray]:
    """Rows x [n, C], beta and log_g [n, Hv] through the layer token by token -> (o [n, Hv, dv], T', W')."""
    o = np.zeros((x.shape[0], d.Hv, d.dv))
    for t in range(x.shape[0]):
        T, W, o[t], _, _ = O.token_step(T, W, x[t], beta[t], log_g[t], conv_w, d)
    return o, T, W


def run_batch(lens: Sequence[int], T: np.ndarray, W: np.ndarray, x, beta, log_g, conv_w, d: O.Dims):
    """The rows of a ragged batch, one request after another -> (o [rows, Hv, dv], T' [B, ...], W' [B, ...]); requests
    without rows keep theirs."""
    o, T, W, at = [], T.copy(), W.copy(), 0
    for b, n in enumerate(lens):
        s = slice(at, at + n)
        y, T[b], W[b] = run_sequence(T[b], W[b], x[s], beta[s], log_g[s], conv_w, d)
        o.append(y)
        at += n
    return np.concatenate(o), T, W


def chunk_step(T: np.ndarray, q: np.ndarray, k: np.ndarray, v: np.ndarray, beta: np.ndarray, log_g: np.ndarray):
    """One head's chunk of n tokens in the chunked form: T [dk, dv], q and k [n, dk], v [n, dv] -> (o [n, dv], T').

    With D_ij the product of the gates of tokens j + 1 .. i:  A = (beta_i D_ij k_i.k_j)_{j < i},  M = (1 + A)^-1 diag(beta),
    N = (D_ij q_i.k_j)_{j <= i} M,  w = v - (gates 0 .. i) k T,  u = M w,  o = (gates 0 .. i) q T + N w,
    T' = (all gates) T + k^T (gates i + 1 .. n - 1) u."""
    n = q.shape[0]
    D = np.zeros((n, n))
    for i in range(n):
        for j in range(i + 1):
            D[i, j] = math.exp(log_g[j + 1:i + 1].sum())
    first = np.exp([log_g[:i + 1].sum() for i in range(n)])[:, None]
    last = D[n - 1][:, None]
    A = np.tril(beta[:, None] * D * (k @ k.T), -1)
    M = np.linalg.solve(np.eye(n) + A, np.diag(beta))
    N = (D * (q @ k.T)) @ M
    w = v - first * (k @ T)
    return first * (q @ T) + N @ w, first[n - 1, 0] * T + k.T @ (last * (M @ w))


def log_probabilities(row: np.ndarray) -> np.ndarray:
    m = float(row.max())
    return row - (m + math.log(math.fsum(math.exp(z - m) for z in row.tolist())))


def best_tokens(row: np.ndarray, top: int) -> List[int]:
    """The largest logits' indices, the lower index on ties."""
    return sorted(range(len(row)), key=lambda i: (-row[i], i))[:top]


def entropy(row: np.ndarray) -> float:
    logp = log_probabilities(row)
    return -math.fsum(math.exp(l) * l for l in logp.tolist() if l > -math.inf)
