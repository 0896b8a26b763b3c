"""A bounded cache: attention over all of it, accumulated weights, eviction.

Test infrastructure only (see ``oracle/__init__.py``).  No counterpart on the
pages; the definitions are readings R14-R16 of include/csa2.h.

* visible keys: a token sees the entries whose last token is at or before its own
  position (a token of the prefix: below the prefix's end), the window rows
  max(0, t-W+1) .. t, and with a document mask only keys whose tokens all lie
  in its document.  An eviction moves entries, so their positions say which they
  are (``visible``); entries in order lie at 4 (j + shift) + 3 (``visible_count``);
* logits: tau q.k, capped as cap * tanh(. / cap), minus slope_h |t - p|;
* weights: decay * old + sum over tokens and heads of exp(logit - lse);
* eviction: first n_sink and newest n_recent positions stay, then the highest
  weights (ties: lower index); survivors above ``keep`` fill the holes below.
"""
from __future__ import annotations

import numpy as np


def visible_count(n_entries: int, shift: int, t: int, prefix_len: int = 0) -> int:
    """Entries in order: 0 .. count-1 are those that the token at raw position t may see (before a document mask)."""
    if t < 0:
        return 0
    sees = max(t + 1, prefix_len) if t < prefix_len else t + 1   # raw tokens 0 .. sees-1
    count = 0
    done = sees // 4 - shift          # entries complete within them, less the evicted ones
    if done > 0:
        count = min(done, n_entries)
    return count


def visible(pos: np.ndarray, t: int, prefix_len: int = 0) -> np.ndarray:
    """Indices of the entries, their last tokens at raw positions pos, that the token at raw position t may see."""
    if t < 0:
        return np.zeros(0, np.int64)
    return np.flatnonzero(np.asarray(pos, np.int64) <= max(t, prefix_len - 1))


def logits(q: np.ndarray, keys: np.ndarray, tau: float, t: int, pos: np.ndarray, cap: float = 0.0, slopes=None):
    """Logits [Hq, n] of one token's heads q [Hq, d] against keys [n, d] at raw positions pos [n]."""
    x = np.asarray(q, np.float64) @ np.asarray(keys, np.float64).T * tau
    if cap > 0:
        x = cap * np.tanh(x / cap)
    if slopes is not None:
        x = x - np.asarray(slopes, np.float64)[:, None] * np.abs(t - np.asarray(pos, np.float64))[None, :]
    return x


def attention(x: np.ndarray, keys: np.ndarray):
    """(O, lse) of logits x [Hq, n] over values = keys [n, d]; no key: zeros and -inf."""
    if x.shape[1] == 0:
        return np.zeros((x.shape[0], keys.shape[1])), np.full(x.shape[0], -np.inf)
    m = x.max(axis=1, keepdims=True)
    e = np.exp(x - m)
    l = e.sum(axis=1, keepdims=True)
    return (e / l) @ np.asarray(keys, np.float64), (m + np.log(l))[:, 0]


def evict(weight: np.ndarray, pos: np.ndarray, shift: int, keep: int, n_sink: int, n_recent: int):
    """(holes, movers): the i-th survivor at an index >= keep goes to the i-th evicted index < keep."""
    n = len(weight)
    if n <= keep:
        return np.zeros(0, np.int64), np.zeros(0, np.int64)
    entry = np.asarray(pos, np.int64) // 4                     # number of the entry since the sequence began
    always = (entry < n_sink) | (entry >= n + shift - n_recent)
    order = sorted(range(n), key=lambda j: (not always[j], -float(weight[j]) if not always[j] else 0.0, j))
    stays = np.zeros(n, bool)
    stays[order[:keep]] = True
    j = np.arange(n)
    return j[(j < keep) & ~stays], j[(j >= keep) & stays]
