"""The 8-bit cache's oracle against values worked out by hand."""

import math

import numpy as np
import pytest

from oracle import fp8
from tests.fp8_support import write_many


@pytest.mark.parametrize("xs, e", [
    ([448.0], 127), ([448.5], 128), ([449.0, -3.0], 128), ([1.75], 119), ([1.7500001], 120), ([1.0], 119),
    ([0.0, -0.0], 10), ([math.nan, 2.0, math.inf], 120), ([1e-45], 10), ([3.4e38], 246), ([math.nan], 10)])
def test_scale(xs, e):
    assert fp8.scale_of(xs) == e


@pytest.mark.parametrize("x, e, c", [
    (1.0, 127, 0x38), (-1.0, 127, 0xB8), (448.0, 127, 0x7E), (1e9, 127, 0x7E), (-1e9, 127, 0xFE),
    (2.0 ** -9, 127, 1), (2.0 ** -10, 127, 0), (1.0001 * 2.0 ** -10, 127, 1), (3 * 2.0 ** -10, 127, 2),
    (1.0625, 127, 0x38), (1.1875, 127, 0x3A), (-0.0, 127, 0x80), (math.nan, 127, 0x7F), (-math.inf, 127, 0x7F),
    (1.0, 119, 0x78), (464.0, 127, 0x7E)])
def test_code(x, e, c):
    assert fp8.code(x, e) == c
    if c not in (0x7F, 0x7E, 0xFE):
        assert abs(fp8.value(c, e) - x) <= max(abs(x) * 2.0 ** -4, 2.0 ** (e - 127 - 10))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("is_key", [True, False])
def test_places_are_a_permutation(d, is_key):
    at = {fp8.place(t, i, d, is_key) for t in range(16) for i in range(d)}
    assert at == set(range(16 * d))


def test_a_block_fills_and_begins_anew():
    d = 64
    pool = np.full((2, fp8.chunk_bytes(d)), 0xAB, np.uint8)
    one = np.ones((1, 1, d))
    fp8.write(pool, [16], one, True)              # row 0 of block 1: the rest becomes zero
    assert pool[1, 16 * d] == 119 and (pool[1, 16 * d + 1:] == 0).all() and (pool[0] == 0xAB).all()
    rows = fp8.read_rows(pool, np.arange(16, 32), 1, d, True)
    assert (rows[0] == 1).all() and (rows[1:] == 0).all()
    fp8.write(pool, [18], one * 2.0 ** -12, True)      # fits below: the scale stays
    assert pool[1, 16 * d] == 119
    # grows by 2^6: 100 is code 400, between 384 (even) and 416; 2^-12 half the least code's step
    fp8.write(pool, [17], one * 100, True)
    rows = fp8.read_rows(pool, np.arange(16, 32), 1, d, True)
    assert pool[1, 16 * d] == 125 and (rows[0] == 1).all() and (rows[1] == 96).all()
    assert (rows[2] == 0).all()
    fp8.write(pool, [16, 16], np.concatenate([one, 3 * one]), True)     # the last of two
    rows = fp8.read_rows(pool, np.arange(16, 32), 1, d, True)
    assert (rows[0] == 3).all() and (rows[1:] == 0).all() and pool[1, 16 * d] == 120


def test_tables():
    none = fp8.cos_sin(5, 8)
    assert none[0].tolist() == [1, 1, 1, 1, 0, 0, 0, 0]
    assert none[3, 0] == math.cos(3.0) and none[3, 4] == math.sin(3.0)
    assert np.allclose(none[3, 1], math.cos(0.3), atol=1e-15)
    assert np.allclose(fp8.cos_sin(2, 8, scaling="linear", factor=4.0, start=8)[0], fp8.cos_sin(3, 8)[2])
    # both ends of the ramps: what turns often stays, what turns seldom is interpolated
    f, p = (fp8.frequencies(64, 1e4, s, 8.0, 4096, 1.0, 32.0) for s in ("parts", "yarn"))
    w = fp8.frequencies(64, 1e4, "none", 1.0, 0, 0, 0)
    assert f[0] == w[0] == p[0] and f[-1] == w[-1] / 8 and p[-1] == w[-1] / 8
    assert np.isclose(fp8.frequencies(64, 1e4, "ntk", 8.0, 0, 0, 0)[-1], w[-1] / 8)


@pytest.mark.parametrize("is_key", [True, False])
@pytest.mark.parametrize("d", [64, 128])
def test_writes_of_whole_arrays_are_those_of_single_values(d, is_key):
    rng = np.random.default_rng(d)
    pools = [rng.integers(0, 256, (6, 2 * fp8.chunk_bytes(d)), dtype=np.uint8)]
    pools.append(pools[0].copy())
    for call in range(3):
        slots = rng.integers(-1, 96, 30)
        rows = rng.standard_normal((30, 2, d)) * np.exp2(rng.integers(-30, 30, (30, 2, 1)))
        rows[3] = 0.0
        rows[4, 0, :5] = np.nan, np.inf, -np.inf, -0.0, 464.0
        rows[5] = rng.choice(np.concatenate([fp8.TABLE[:127], (fp8.TABLE[1:127] + fp8.TABLE[:126]) / 2]), (2, d))
        fp8.write(pools[0], slots, rows, is_key)
        write_many(pools[1], slots, rows, is_key)
        assert np.array_equal(*pools)
