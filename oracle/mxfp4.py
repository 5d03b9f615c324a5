"""The 4-bit paged cache and the device-built step metadata, plainly.

Everything here is one value at a time, in exact arithmetic where it matters:

* `quantise`      - one group of 32 numbers to (scale byte, codes): the scale is
                    the power of two that brings the largest magnitude into
                    [4, 8), each code the nearest number of the e2m1 grid, of
                    two equally near the one with the even code
* `value`         - the number a (code, scale byte) pair stands for
* `code_place`,
  `scale_place`   - where the code and the scale of a dimension sit in a block
* `step_metadata` - block tables, slots and positions of a step, a token at a
                    time, taking a block from the ring whenever a token starts one
"""

from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

BLOCK = 16
GROUP = 32
GRID = [Fraction(x) for x in ("0", "1/2", "1", "3/2", "2", "3", "4", "6")]


def _floor_log2(x: Fraction) -> int:
    k = x.numerator.bit_length() - x.denominator.bit_length()
    while Fraction(2) ** k > x:
        k -= 1
    while Fraction(2) ** (k + 1) <= x:
        k += 1
    return k


def quantise(group) -> tuple[int, list[int]]:
    """(scale byte, codes) of 32 floats."""
    xs = [float(x) for x in group]
    if not all(math.isfinite(x) for x in xs):
        return 255, [0] * len(xs)
    amax = max(abs(Fraction(x)) for x in xs)
    if amax == 0:
        e = 127
    else:
        e = min(254, max(1, _floor_log2(amax) - 2 + 127))
    codes = []
    for x in xs:
        y = abs(Fraction(x)) / Fraction(2) ** (e - 127)
        best = min(range(8), key=lambda i: (abs(y - GRID[i]), i % 2))
        codes.append(best + (8 if math.copysign(1.0, x) < 0 else 0))
    return e, codes


def value(code: int, e: int) -> float:
    if e == 255:
        return math.nan
    v = float(GRID[code % 8]) * 2.0 ** (e - 127)
    return -v if code >= 8 else v


def chunk_bytes(d: int) -> int:
    """Bytes of one KV head in one block."""
    return BLOCK * d // 2 + BLOCK * d // GROUP


def code_place(t: int, dim: int, d: int, is_key: bool) -> tuple[int, int]:
    """(byte within the head's chunk, 0 for the low nibble or 1) of a code."""
    b, w = divmod(dim, 32)
    if is_key:
        byte = (w // 8) * (d // 8) + 4 * b + (w % 8) // 2
    else:
        byte = (w // 4) * (d // 16) + 2 * b + (w % 4) // 2
    return t * (d // 2) + byte, dim % 2


def scale_place(t: int, b: int, d: int, is_key: bool) -> int:
    """Byte within the head's chunk of the scale of group b of token t."""
    if is_key:
        return BLOCK * d // 2 + t * (d // 32) + b
    return BLOCK * d // 2 + (t // 2) * (d // 16) + (b // 2) * 4 + (t % 2) * 2 + b % 2


def write_row(pool: np.ndarray, slot: int, row: np.ndarray, is_key: bool) -> None:
    """Quantise row [Hkv, D] into pool (uint8 [num_blocks, block bytes]) at slot."""
    hkv, d = row.shape
    blk, t = divmod(slot, BLOCK)
    for h in range(hkv):
        base = h * chunk_bytes(d)
        for b in range(d // GROUP):
            e, codes = quantise(row[h, b * GROUP:(b + 1) * GROUP])
            pool[blk, base + scale_place(t, b, d, is_key)] = e
            for i, c in enumerate(codes):
                byte, high = code_place(t, b * GROUP + i, d, is_key)
                old = int(pool[blk, base + byte])
                pool[blk, base + byte] = (old & 0x0f) | c << 4 if high else (old & 0xf0) | c


_VALUES = np.array([[value(c, e) for c in range(16)] for e in range(256)])


def read_rows(pool: np.ndarray, slots, hkv: int, d: int, is_key: bool) -> np.ndarray:
    """float64 [n, Hkv, D] of the values at slots."""
    out = np.empty((len(slots), hkv, d))
    place = [[code_place(t, i, d, is_key) + (scale_place(t, i // GROUP, d, is_key),)
              for i in range(d)] for t in range(BLOCK)]
    place = np.array(place)  # [16, D, (byte, nibble, scale byte)]
    for n, s in enumerate(slots):
        blk, t = divmod(int(s), BLOCK)
        for h in range(hkv):
            chunk = pool[blk, h * chunk_bytes(d):(h + 1) * chunk_bytes(d)]
            byte = chunk[place[t, :, 0]].astype(np.int64)
            code = np.where(place[t, :, 1] == 1, byte >> 4, byte & 15)
            out[n, h] = _VALUES[chunk[place[t, :, 2]], code]
    return out


class Refused(Exception):
    """The step is refused whole; args[0] is "metadata" or "blocks"."""


def step_metadata(query_lens, num_computed, table, ring, head: int, tail: int, num_tokens: int):
    """(table, query_start_loc, seq_lens, slots, positions, head) after the step.
    table is a list of rows of equal length; raises Refused and changes nothing
    if the step does not fit."""
    width = len(table[0]) if table else 0
    if head < 0 or tail < head or tail - head > len(ring):
        raise Refused("metadata")
    for s, n in zip(query_lens, num_computed):
        if s < 0 or n < 0 or -(-(n + s) // BLOCK) > width:
            raise Refused("metadata")
    if sum(query_lens) > num_tokens:
        raise Refused("metadata")
    need = sum(-(-(n + s) // BLOCK) - -(-n // BLOCK) for s, n in zip(query_lens, num_computed))
    if need > tail - head:
        raise Refused("blocks")
    table = [list(r) for r in table]
    qsl, slots, positions = [0], [], []
    for r, (s, n) in enumerate(zip(query_lens, num_computed)):
        for p in range(n, n + s):
            if p % BLOCK == 0:
                table[r][p // BLOCK] = ring[head % len(ring)]
                head += 1
            blk = table[r][p // BLOCK]
            slots.append(blk * BLOCK + p % BLOCK if blk >= 0 else -1)
            positions.append(p)
        qsl.append(len(slots))
    fill = num_tokens - len(slots)
    return (table, qsl, [n + s for s, n in zip(query_lens, num_computed)], slots + [-1] * fill,
            positions + [0] * fill, head)
