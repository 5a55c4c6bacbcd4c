"""The 8-bit paged cache in float64, from its definition: a row's exponent byte,
its e4m3 codes, what they stand for, and the commit of a tree's path.  Test
infrastructure; shares no code with the library."""
import math
from typing import Optional

import numpy as np

# values of the codes 0x00 .. 0x7e: e = 0: m * 2^-9, else (8 + m) * 2^(e - 10); 0x7f is NaN
E4M3 = np.array([(m * 2.0 ** -9) if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)])
E4M3[127] = np.nan


def kv8_quantise(x):
    """(codes uint8 [..., D], scale uint8 [...]) of rows x [..., D]."""
    x = np.asarray(x, np.float64)
    codes, scale = np.zeros(x.shape, np.uint8), np.zeros(x.shape[:-1], np.uint8)
    for at in np.ndindex(*x.shape[:-1]):
        row = x[at]
        if not np.isfinite(row).all():
            scale[at] = 255
            continue
        top, s = np.abs(row).max(), 1
        if top > 0:
            s = max(1, math.ceil(math.log2(top / 448.0) - 1e-9) + 127)
            while top > 448.0 * 2.0 ** (s - 127):
                s += 1
            while s > 1 and top <= 448.0 * 2.0 ** (s - 128):
                s -= 1
        scale[at] = s
        y = np.abs(row) * 2.0 ** (127 - s)
        lo = np.clip(np.searchsorted(E4M3[:127], y, side="right") - 1, 0, 126)
        hi = np.minimum(lo + 1, 126)
        below, above = y - E4M3[lo], E4M3[hi] - y
        up = (above < below) | ((above == below) & (lo % 2 == 1))    # ties: the even code
        codes[at] = np.where(up, hi, lo) | np.where(np.signbit(row), 128, 0)
    return codes, scale


def kv8_values(codes, scale):
    """float64 [..., D] of codes uint8 [..., D] and scale uint8 [...]."""
    codes, scale = np.asarray(codes, np.int64), np.asarray(scale, np.int64)
    power = np.where(scale == 255, np.nan, 2.0 ** (scale - 127.0))
    return np.where(codes >= 128, -1.0, 1.0) * E4M3[codes & 127] * power[..., None]


def kv8_commit(codes, scale, table, block_size, length, slots, S) -> Optional[int]:
    """Moves one request's kept candidates, in place (codes [L, 2, nb, bs, H, D],
    scale [L, 2, nb, H, bs]); the new length, or None for bad data."""
    n, nb, capacity = len(slots), codes.shape[2], len(table) * block_size
    if length < 0 or n > S or length + n > capacity:
        return None
    if any(s < 0 or s >= S for s in slots) or any(b <= a for a, b in zip(slots, slots[1:])):
        return None
    moves = [(length + s, length + i) for i, s in enumerate(slots) if s != i]
    if any(a >= capacity for a, _ in moves) or any(not 0 <= table[x // block_size] < nb for m in moves for x in m):
        return None
    for a, b in moves:
        (sa, oa), (sb, ob) = ((table[x // block_size], x % block_size) for x in (a, b))
        codes[:, :, sb, ob] = codes[:, :, sa, oa]
        scale[:, :, sb, :, ob] = scale[:, :, sa, :, oa]
    return length + n
