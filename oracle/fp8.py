"""The 8-bit paged cache and the table of rotary angles, plainly.

Everything here is one value at a time, in exact arithmetic where it matters:

* `scale_of`   - the scale byte of some numbers: the smallest power of two that keeps
                 the largest finite magnitude within 448, the largest e4m3 number
* `code`       - the nearest e4m3 code of a number at a scale, of two equally near the
                 even one
* `value`      - the number a (code, scale byte) pair stands for
* `place`      - where the code of a token and dimension sits in a KV head's chunk
* `write`      - a call's rows into a pool, a block at a time
* `cos_sin`    - the table of rotary angles with its long-context scalings
"""

from __future__ import annotations

import bisect
import math
from fractions import Fraction

import numpy as np

BLOCK = 16
NAN = 0x7F
LOW, HIGH = 10, 246
# magnitudes of the codes 0 .. 126, ascending
GRID = [Fraction(m, 512) if e == 0 else Fraction(8 + m, 8) * Fraction(2) ** (e - 7)
        for e in range(16) for m in range(8)][:NAN]
TABLE = np.array([float(g) for g in GRID] + [math.nan])
TABLE = np.concatenate([TABLE, -TABLE])


def clamped(e: int) -> int:
    return min(max(int(e), LOW), HIGH)


def scale_of(xs) -> int:
    most = max((abs(Fraction(float(x))) for x in xs if math.isfinite(x)), default=Fraction(0))
    e = LOW
    while e < HIGH and most > 448 * Fraction(2) ** (e - 127):
        e += 1
    return e


def code(x: float, e: int) -> int:
    x = float(x)
    if not math.isfinite(x):
        return NAN
    y = abs(Fraction(x)) / Fraction(2) ** (e - 127)
    hi = min(bisect.bisect_left(GRID, y), NAN - 1)
    best = min((i for i in (hi - 1, hi) if i >= 0), key=lambda i: (abs(y - GRID[i]), i % 2))
    return best + (128 if math.copysign(1.0, x) < 0 else 0)


def value(c: int, e: int) -> float:
    return float(TABLE[c]) * 2.0 ** (clamped(e) - 127)


def chunk_bytes(d: int) -> int:
    """Bytes of one KV head in one block."""
    return BLOCK * d + 16


def place(t: int, dim: int, d: int, is_key: bool) -> int:
    """Byte within the head's chunk of a code."""
    if is_key:
        return ((t // 8) * (d // 64) + dim // 64) * 512 + (t % 8) * 64 + dim % 64
    p = d // 8
    return (dim % p) // 4 * 512 + (dim // p * 4 + (t % 8) // 2) * 16 + dim % 4 * 4 + (t // 8) * 2 + t % 2


def write(pool: np.ndarray, slots, rows: np.ndarray, is_key: bool) -> None:
    """Rows [T, Hkv, D] (float64) to their slots of pool (uint8 [num_blocks, block bytes]);
    negative slots are padding, of a slot given twice the last row counts."""
    _, hkv, d = rows.shape
    blocks: dict[int, dict[int, int]] = {}
    for t, s in enumerate(slots):
        if s >= 0:
            blocks.setdefault(int(s) // BLOCK, {})[int(s) % BLOCK] = t
    for blk, new in blocks.items():
        for h in range(hkv):
            chunk = pool[blk, h * chunk_bytes(d):(h + 1) * chunk_bytes(d)]
            e = scale_of(np.concatenate([rows[t, h] for t in new.values()]))
            old = None if 0 in new else clamped(chunk[BLOCK * d])
            if old is not None:
                e = max(e, old)
            for off in range(BLOCK):
                for dim in range(d):
                    at = place(off, dim, d, is_key)
                    if off in new:
                        chunk[at] = code(rows[new[off], h, dim], e)
                    elif old is None:
                        chunk[at] = 0
                    elif e > old:
                        c = int(chunk[at])
                        again = code(float(TABLE[c % 128]) * 2.0 ** (old - e), 127) if c % 128 != NAN else NAN
                        chunk[at] = again + c // 128 * 128 if again != NAN else NAN
            chunk[BLOCK * d:] = 0
            chunk[BLOCK * d] = e


def read_rows(pool: np.ndarray, slots: np.ndarray, hkv: int, d: int, is_key: bool) -> np.ndarray:
    """float64 [len(slots), Hkv, D]."""
    out = np.empty((len(slots), hkv, d))
    at = np.array([[place(t, i, d, is_key) for i in range(d)] for t in range(BLOCK)])
    for h in range(hkv):
        base = h * chunk_bytes(d)
        c = pool[(slots // BLOCK)[:, None], base + at[slots % BLOCK]]
        e = np.clip(pool[slots // BLOCK, base + BLOCK * d].astype(np.int64), LOW, HIGH)
        out[:, h] = TABLE[c] * np.exp2(e - 127.0)[:, None]
    return out


def frequencies(rd: int, base: float, scaling: str, factor: float, length: int, low: float, high: float):
    """The rd / 2 frequencies, radians a position."""
    out = []
    for i in range(rd // 2):
        w = base ** (-2 * i / rd)
        if scaling == "linear":
            w /= factor
        elif scaling == "ntk":
            w = (base * factor ** (rd / (rd - 2))) ** (-2 * i / rd)
        elif scaling == "parts":
            turns = length * w / (2 * math.pi)
            g = 0.0 if turns <= low else 1.0 if turns >= high else (turns - low) / (high - low)
            w = g * w + (1 - g) * w / factor
        elif scaling == "yarn":
            a = max(0, math.floor(rd * math.log(length / (2 * math.pi * high)) / (2 * math.log(base))))
            b = min(rd - 1, math.ceil(rd * math.log(length / (2 * math.pi * low)) / (2 * math.log(base))))
            g = 1 - min(1.0, max(0.0, (i - a) / max(b - a, 0.001)))
            w = g * w + (1 - g) * w / factor
        out.append(w)
    return out


def cos_sin(n: int, rd: int, base=10000.0, scaling="none", factor=1.0, length=0, low=1.0, high=32.0,
            attention=1.0, start=0) -> np.ndarray:
    """float64 [n, rd]."""
    p = np.arange(start, start + n, dtype=np.float64)[:, None]
    angle = p * np.array(frequencies(rd, base, scaling, factor, length, low, high))
    return attention * np.concatenate([np.cos(angle), np.sin(angle)], 1)
