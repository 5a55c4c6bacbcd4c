"""Attention over the paged cache, entry weights and eviction in float64, one
request at a time, from their definitions.  Test infrastructure; shares no
code with the library."""
import math
from dataclasses import dataclass
from typing import Optional

import numpy as np


def entries(plane, table, block_size, n):
    """Rows [n, H, D] of a layer's plane [num_blocks, block_size, H, D] for the
    first n entries of one request."""
    return np.array([plane[table[c // block_size], c % block_size] for c in range(n)], np.float64).reshape(
        (n,) + plane.shape[2:])


def scores(q, k, q_pos, k_pos, *, scale, softcap=0.0, slopes=None):
    """[Hq, S, N] of q [S, Hq, D] against k [N, H, D]."""
    S, Hq, D = q.shape
    H = k.shape[1]
    x = np.empty((Hq, S, k.shape[0]))
    dist = np.asarray(q_pos, np.float64)[:, None] - np.asarray(k_pos, np.float64)[None, :]
    for h in range(Hq):
        x[h] = scale * (q[:, h].astype(np.float64) @ k[:, h // (Hq // H)].T)
        if softcap:
            x[h] = softcap * np.tanh(x[h] / softcap)
        if slopes is not None:
            x[h] -= float(slopes[h]) * dist
    return x


def hidden(q_pos, k_pos, *, first_pos=None, window=0):
    """[S, N]: masked by position."""
    dist = np.asarray(q_pos, np.int64)[:, None] - np.asarray(k_pos, np.int64)[None, :]
    m = np.zeros(dist.shape, bool)
    if window:
        m |= dist >= window
    if first_pos is not None:
        m |= (np.asarray(k_pos, np.int64) < first_pos)[None, :]
    return m


@dataclass
class Attention:
    out: np.ndarray      # [S, Hq, D]
    lse: np.ndarray      # [S, Hq]
    p: np.ndarray        # [Hq, S, N]
    mass: np.ndarray     # [S, Hq, D]: sum of p |v|


def attend(q, k, v, q_pos, k_pos, masked, **score):
    """Softmax attention of q [S, Hq, D]; masked [S, N]."""
    S, Hq, D = q.shape
    H = k.shape[1]
    x = scores(q, k, q_pos, k_pos, **score)
    x = np.where(masked[None], -np.inf, x)
    out, mass = np.zeros((S, Hq, D)), np.zeros((S, Hq, D))
    lse, p = np.full((S, Hq), -np.inf), np.zeros(x.shape)
    for h in range(Hq):
        vh = v[:, h // (Hq // H)].astype(np.float64)
        for i in range(S):
            seen = ~masked[i]
            if not seen.any():
                continue
            m = x[h, i, seen].max()
            e = np.exp(x[h, i, seen] - m)
            lse[i, h] = m + math.log(e.sum())
            p[h, i, seen] = e / e.sum()
            out[i, h] = p[h, i, seen] @ vh[seen]
            mass[i, h] = p[h, i, seen] @ np.abs(vh[seen])
    return Attention(out, lse, p, mass)


def candidate_mask(S, words=None):
    """[S, S]: candidate j masked for candidate i (words: the tree mask)."""
    m = np.ones((S, S), bool)
    for i in range(S):
        for j in range(S):
            seen = j <= i if words is None else (int(words[i][j // 32]) & 0xFFFFFFFF) >> (j % 32) & 1
            m[i, j] = not seen
    return m


def entry_weights(q, lse, k, q_pos, k_pos, n, *, first_pos=None, window=0, start=0, **score):
    """What the entries [len(k)] gain: q [n, Hq, D] and lse [n, Hq] are the
    committed candidates', the last n entries their own."""
    L = k.shape[0]
    x = scores(q, k, q_pos, k_pos, **score)
    off = hidden(q_pos, k_pos, first_pos=first_pos, window=window)
    gain = np.zeros(L)
    for j in range(n):
        for c in range(start, L - n + j + 1):
            if off[j, c]:
                continue
            for h in range(q.shape[1]):
                if lse[j, h] > -np.inf:
                    gain[c] += math.exp(x[h, j, c] - lse[j, h])
    return gain


@dataclass
class Eviction:
    kept: list           # entries kept, ascending
    moves: list          # (from, to)
    length: int


def evict(weight, pos, length, *, budget, sink=0, recent=0) -> Optional[Eviction]:
    """None: the request's data are bad."""
    w, p = list(map(float, weight[:length])), list(map(int, pos[:length]))
    if length <= budget:
        return Eviction(list(range(length)), [], length)
    if any(math.isnan(x) for x in w) or any(x < 0 for x in p):
        return None
    newest = max(p)
    safe = [c for c in range(length) if p[c] < sink or p[c] > newest - recent]
    if len(safe) > budget:
        return None
    protected = set(safe)
    others = sorted((c for c in range(length) if c not in protected), key=lambda c: (-w[c], c))
    kept = sorted(safe + others[:budget - len(safe)])
    holes = sorted(set(range(budget)) - set(kept))
    return Eviction(kept, list(zip([c for c in kept if c >= budget], holes)), budget)
