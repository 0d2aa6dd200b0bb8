"""Normed rows, block scores, the choice of blocks and attention over chosen blocks in numpy, 64 bits, from their
definitions.  Shares no code with the CUDA path.  A block is 64 positions."""
from __future__ import annotations

import numpy as np

from oracle import paged_oracle as PO

BLOCK = 64


def rms(x: np.ndarray, weight, eps: float) -> np.ndarray:
    """x [.., n] over the root of its mean square, times weight [n] (None: x as it is)."""
    if weight is None:
        return x.astype(np.float64)
    x = x.astype(np.float64)
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight


def mean_rows(rows: np.ndarray) -> np.ndarray:
    """[n, 576] -> the mean rows of its n // 64 whole blocks."""
    n = rows.shape[0] // BLOCK
    return rows[:n * BLOCK].reshape(n, BLOCK, rows.shape[1]).mean(1)


def block_scores(q: np.ndarray, keys: np.ndarray, p0: int, width: int, scale: float):
    """q [n, H, 576] at positions p0, p0 + 1, ..; keys [m, 576] -> (scores [n, width], the largest sum of |products| [n,
    width])."""
    out, mag = np.full((q.shape[0], width), -np.inf), np.zeros((q.shape[0], width))
    for i in range(q.shape[0]):
        k = min((p0 + i) // BLOCK, width)
        if k:
            out[i, :k] = scale * (q[i] @ keys[:k].T).max(0)
            mag[i, :k] = scale * (np.abs(q[i]) @ np.abs(keys[:k]).T).max(0)
    return out, mag


def select(scores: np.ndarray, p: int, K: int, n_sink: int, n_local: int) -> np.ndarray:
    """The blocks that a token at position p takes, ascending."""
    own = p // BLOCK
    forced = {j for j in range(own + 1) if j < n_sink or j > own - n_local}
    rest = [j for j in range(own) if j not in forced]
    # NaN below everything; Python's sort is stable: equal scores stay in order
    rest.sort(key=lambda j: (np.isnan(scores[j]), 0.0 if np.isnan(scores[j]) else -float(scores[j])))
    return np.array(sorted(forced | set(rest[:K - len(forced)])), np.int32)


def attend_blocks(q: np.ndarray, rows: np.ndarray, p: int, blocks, scale: float):
    """q [H, 576] at position p over the listed blocks' rows (a block as often as it is listed) ->
    (o [H, 512], sum_j p_j |c_j| [H, 512], the number of keys seen)."""
    keys = np.concatenate([np.arange(64 * b, min(64 * b + 64, p + 1)) for b in blocks]) if len(blocks) else np.zeros(0, int)
    if len(keys) == 0:
        return np.zeros((q.shape[0], PO.LAT)), np.zeros((q.shape[0], PO.LAT)), 0
    s = scale * (q @ rows[keys].T)
    w = np.exp(s - s.max(-1, keepdims=True))
    w /= w.sum(-1, keepdims=True)
    return w @ rows[keys, :PO.LAT], w @ np.abs(rows[keys, :PO.LAT]), len(keys)
