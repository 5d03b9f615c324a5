"""Pins of the 4-bit cache's oracle and of the device step metadata's oracle."""

import math
import random

import numpy as np
import pytest

from oracle import mxfp4, paging
from oracle.allocator import NaiveAllocator


def _group(first, rest=0.0):
    return [first] + [rest] * 31


@pytest.mark.parametrize("x, code", [(0.25, 0), (0.26, 1), (0.75, 2), (0.74, 1), (1.25, 2),
                                     (1.26, 3), (1.75, 4), (2.5, 4), (2.51, 5), (3.5, 6),
                                     (5.0, 6), (5.01, 7), (6.0, 7), (7.99, 7)])
def test_rounding_ties_to_even_codes_and_saturation(x, code):
    # 4 (or more) in the group fixes the scale at 1
    e, codes = mxfp4.quantise([x, -x, max(4.0, x)] + [0.0] * 29)
    assert e == 127
    assert codes[:2] == [code, code + 8]


@pytest.mark.parametrize("amax, e", [(1.0, 125), (1.99, 125), (2.0, 126), (4.0, 127), (7.99, 127),
                                     (8.0, 128), (2.0 ** -126, 1), (2.0 ** -149, 1),
                                     (3.38e38, 252), (0.0, 127)])
def test_scale_byte(amax, e):
    assert mxfp4.quantise(_group(amax))[0] == e


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_non_finite_group_is_nan(bad):
    e, codes = mxfp4.quantise(_group(bad, 1.0))
    assert e == 255 and codes == [0] * 32
    assert all(math.isnan(mxfp4.value(c, e)) for c in codes)


def test_values():
    assert [mxfp4.value(c, 127) for c in range(8)] == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert [mxfp4.value(c + 8, 129) for c in range(1, 8)] == [-2, -4, -6, -8, -12, -16, -24]
    assert mxfp4.value(7, 0) == 6 * 2.0 ** -127


def test_quantisation_error_bound():
    """Half a grid step: at most amax / 8 for the large half of the grid (its
    step is 2 of an amax in [4, 8)), and saturation takes off less than 2."""
    rng = np.random.default_rng(0)
    for _ in range(50):
        g = rng.standard_normal(32) * 2.0 ** rng.integers(-20, 20)
        e, codes = mxfp4.quantise(g)
        err = max(abs(x - mxfp4.value(c, e)) for x, c in zip(g, codes))
        assert err <= 2.0 * 2.0 ** (e - 127)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("is_key", [True, False])
def test_layout_is_a_bijection(d, is_key):
    codes = {mxfp4.code_place(t, i, d, is_key) for t in range(16) for i in range(d)}
    assert codes == {(b, n) for b in range(8 * d) for n in (0, 1)}
    scales = {mxfp4.scale_place(t, b, d, is_key) for t in range(16) for b in range(d // 32)}
    assert scales == set(range(8 * d, mxfp4.chunk_bytes(d)))


@pytest.mark.parametrize("is_key", [True, False])
def test_write_then_read_touches_its_rows_only(is_key):
    rng = np.random.default_rng(1)
    pool = rng.integers(0, 256, (3, 2 * mxfp4.chunk_bytes(64)), dtype=np.uint8)
    before = mxfp4.read_rows(pool, range(48), 2, 64, is_key)
    row = rng.standard_normal((2, 64))
    mxfp4.write_row(pool, 21, row, is_key)
    after = mxfp4.read_rows(pool, range(48), 2, 64, is_key)
    others = [i for i in range(48) if i != 21]
    assert np.array_equal(before[others], after[others], equal_nan=True)
    assert np.abs(after[21] - row).max() <= 0.5


def test_step_metadata_agrees_with_the_allocator():
    rng = random.Random(5)
    for _ in range(30):
        n = rng.randint(1, 6)
        pool = 64
        alloc = NaiveAllocator(pool, 16)
        held = [rng.randint(0, 60) for _ in range(n)]
        assert alloc.reserve([(r, h) for r, h in enumerate(held) if h])
        alloc.commit()
        table = [(alloc.table(r) + [-1] * 12)[:12] for r in range(n)]
        ring = list(alloc.free_list)
        new = [rng.randint(0, 40) for _ in range(n)]
        got = mxfp4.step_metadata(new, held, table, ring, 0, len(ring), 300)
        assert alloc.reserve([(r, s) for r, s in enumerate(new) if s])
        rows = [alloc.table(r) for r in range(n)]
        assert [[b for b in row if b >= 0] for row in got[0]] == rows
        assert got[3][:sum(new)] == paging.slot_mapping(rows, new, held, 16)
        assert got[3][sum(new):] == [-1] * (300 - sum(new))
        assert got[2] == [h + s for h, s in zip(held, new)]


@pytest.mark.parametrize("new, held, tokens, tail, why", [
    ([1, -1], [0, 0], 8, 4, "metadata"), ([1], [-3], 8, 4, "metadata"),
    ([40], [0], 64, 4, "metadata"), ([5, 4], [0, 0], 8, 4, "metadata"),
    ([16, 17], [0, 0], 64, 2, "blocks")])
def test_step_metadata_refusals(new, held, tokens, tail, why):
    with pytest.raises(mxfp4.Refused, match=why):
        mxfp4.step_metadata(new, held, [[-1, -1]] * len(new), [7, 8, 9, 10], 0, tail, tokens)
