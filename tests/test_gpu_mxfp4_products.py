"""The 4-bit attention where what a key contributes is not told by its weight or its value
alone: unlikely keys with large values, likely ones with small values, groups of
dimensions far apart.  The bound (tests/mxfp4_bounds.py) goes by weight times value."""

import numpy as np
import pytest
import torch

from oracle import mxfp4
from tests.mxfp4_bounds import check, reference
from tests.mxfp4_support import Step

pytestmark = pytest.mark.gpu

DECODE = [(1, 700), (1, 40), (1, 1500)]
KINDS = {"decode": DECODE, "direct": [(20, 270), (3, 7)], "ahead": [(60, 900)]}


def _attend(s):
    import paged_kv_cache_36_gb300 as pkv
    ws = pkv.new_workspace_mxfp4(s.H, s.hkv, s.d)
    got = pkv.paged_attention_varlen_mxfp4(*s.args(), workspace=ws, max_query_len=max(s.q_len))
    assert pkv.read_error_word(ws) == 0
    return got


def _step(seed, kind, d, octaves, heads=4):
    """Keys whose scores are -octaves(j) in log2 units for even heads, half of that for odd
    ones (octaves: a number of the 4-bit grid, times a power of two)."""
    s = Step(seed, KINDS[kind], heads, 1, d)
    s.q[:, :, :] = 0
    s.q[:, ::2, 0] = 1.0
    s.q[:, 1::2, 0] = 0.5
    s.scale = float(np.log(2.0))
    for slots in s.slots:
        for j, slot in enumerate(slots.tolist()):
            row = np.zeros((1, d))
            row[0, 0] = -octaves(j)
            mxfp4.write_row(s.pools.k, slot, row, True)
    return s


@pytest.mark.parametrize("kind", ["decode"])
@pytest.mark.parametrize("octaves, up", [(24, 24), (32, 40), (32, 24), (48, 48), (96, 90)])
@pytest.mark.parametrize("d", [64, 128])
def test_unlikely_keys_with_large_values(kind, octaves, up, d):
    """Every third key is 2^octaves (or the root of that) less likely than the others, with
    values 2^up times theirs."""
    s = _step(1, kind, d, lambda j: octaves if j % 3 == 0 else 0.25 * (j % 4))
    for slots in s.slots:
        s.pools.scales(s.rng, slots[::3], up - 1, up + 1, k=False)
    s.upload()
    check(_attend(s), *reference(s))


@pytest.mark.parametrize("kind", ["decode"])
@pytest.mark.parametrize("octaves, down", [(12, 12), (24, 24), (24, 40)])
@pytest.mark.parametrize("d", [64, 128])
def test_one_likely_key_with_small_values(kind, octaves, down, d):
    """The first key has most of the weight, and values 2^-down times the others'."""
    s = _step(2, kind, d, lambda j: 0 if j == 0 else octaves)
    for slots in s.slots:
        s.pools.scales(s.rng, slots, -1, 1, k=False)
        s.pools.scales(s.rng, slots[:1], -down, -down, k=False)
    s.upload()
    # even heads; odd ones' weights are the roots
    check(_attend(s), *reference(s), tight=0.6)


@pytest.mark.parametrize("kind", ["decode"])
@pytest.mark.parametrize("octaves", [4, 48])
def test_values_near_the_end_of_float32(kind, octaves):
    """Sums and joins of values of 2^120 stay finite."""
    s = _step(3, kind, 64, lambda j: octaves if j % 3 else 0)
    for slots in s.slots:
        s.pools.scales(s.rng, slots, 120, 122, k=False)
    s.upload()
    check(_attend(s), *reference(s))
