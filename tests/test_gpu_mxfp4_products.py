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


@pytest.mark.parametrize("kind", list(KINDS))
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


@pytest.mark.parametrize("kind", list(KINDS))
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


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("octaves", [4, 48])
def test_values_near_the_end_of_float32(kind, octaves):
    """Sums and joins of values of 2^120 stay finite."""
    s = _step(3, kind, 64, lambda j: octaves if j % 3 else 0)
    for slots in s.slots:
        s.pools.scales(s.rng, slots, 120, 122, k=False)
    s.upload()
    check(_attend(s), *reference(s))


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("which", ["one", "first", "third", "all"])
@pytest.mark.parametrize("above", [20, 30, 40, 70, -30])
@pytest.mark.parametrize("d", [64, 128])
def test_groups_of_dimensions_far_apart(kind, which, above, d):
    """In one key, the first one, a third of them or all of them the first group of dimensions is
    2^above times the others: those keep their own precision."""
    s = Step(4, KINDS[kind], 4, 1, d)
    for slots in s.slots:
        s.pools.scales(s.rng, slots, -1, 1, k=False)
        n = len(slots)
        some = {"one": slice(n // 3, n // 3 + 1), "first": slice(0, 1), "third": slice(0, n, 3),
                "all": slice(0, n)}[which]
        at = slots[some]
        place = np.array([mxfp4.scale_place(t, 0, d, False) for t in range(16)])
        s.pools.v[at // 16, place[at % 16]] = 127 + above
    s.upload()
    check(_attend(s), *reference(s))


@pytest.mark.parametrize("kind", list(KINDS))
def test_groups_of_two_kinds_of_keys(kind):
    """Even keys have their large values in the first group, odd ones in the last."""
    s = Step(5, KINDS[kind], 16, 1, 128)
    for slots in s.slots:
        s.pools.scales(s.rng, slots, -1, 1, k=False)
        for part, group in ((slots[::2], 0), (slots[1::2], 3)):
            place = np.array([mxfp4.scale_place(t, group, 128, False) for t in range(16)])
            s.pools.v[part // 16, place[part % 16]] = 127 + 50
    s.upload()
    check(_attend(s), *reference(s))


def _uneven(s, r, where=slice(None)):
    """Group 0 of the request's values (of some tokens) 2^40 times the others."""
    at = s.slots[r][where]
    for h in range(s.hkv):
        place = np.array([mxfp4.scale_place(t, 0, s.d, False) for t in range(16)])
        s.pools.v[at // 16, place[at % 16] + h * mxfp4.chunk_bytes(s.d)] = 127 + 40


def test_one_request_of_uneven_values_among_others():
    """More query tiles than SMs, the keys that are uneven in the middle of one request."""
    s = Step(6, [(9, 30), (700, 40), (1, 100), (150, 0)], 32, 2, 64)
    _uneven(s, 1, slice(300, 420, 7))
    s.upload()
    check(_attend(s), *reference(s))


@pytest.mark.parametrize("reqs", [[(20, 270), (40, 3)], [(60, 900), (57, 950)]])
def test_uneven_values_leave_nothing_behind(reqs):
    """A workspace through uneven and even batches, captured and replayed."""
    import paged_kv_cache_36_gb300 as pkv
    ws = pkv.new_workspace_mxfp4(16, 1, 64)
    steps = [Step(7 + i, reqs, 16, 1, 64) for i in range(3)]
    _uneven(steps[0], 0)
    _uneven(steps[1], 1, slice(5, 6))
    alone = [_attend(s.upload()) for s in steps]
    for s, a in zip(steps, alone):
        check(a, *reference(s))
    graphs, outs = [], []
    for s in steps:
        out = torch.zeros_like(s.dq)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pkv.paged_attention_varlen_mxfp4(*s.args(), workspace=ws, out=out)
        graphs.append(g)
        outs.append(out)
    for i in (0, 2, 1, 1, 0, 2):
        outs[i].zero_()
        graphs[i].replay()
        assert torch.equal(outs[i], alone[i])
    assert pkv.read_error_word(ws) == 0


@pytest.mark.parametrize("reqs", [[(20, 270)], [(60, 900)]])
def test_nan_among_uneven_values(reqs):
    s = Step(8, reqs, 16, 1, 128)
    _uneven(s, 0, slice(0, None, 5))
    tok = s.past[0] + 7
    slot = int(s.slots[0][tok])
    s.pools.v[slot // 16, mxfp4.scale_place(slot % 16, 2, 128, False)] = 255
    for dim in range(64, 96):
        byte, _ = mxfp4.code_place(slot % 16, dim, 128, False)
        s.pools.v[slot // 16, byte] = 0
    got = _attend(s.upload()).double().cpu()
    ref, tol = reference(s)
    bad = torch.zeros_like(ref, dtype=torch.bool)
    bad[7:, :, 64:96] = True
    assert torch.isnan(got[bad]).all() and torch.isnan(ref[bad]).all()
    assert ((got - ref).abs() <= tol)[~bad].all()


@pytest.mark.parametrize("kind", list(KINDS))
def test_dimensions_that_are_zero(kind):
    """The last group is zero in every token (scale 1, as the cache write leaves it), the
    others' values are 2^-20."""
    s = Step(9, KINDS[kind], 4, 1, 128)
    for slots in s.slots:
        s.pools.scales(s.rng, slots, -21, -19, k=False)
        for t in range(16):
            at = slots[slots % 16 == t] // 16
            s.pools.v[at, mxfp4.scale_place(t, 3, 128, False)] = 127
            for dim in range(96, 128):
                s.pools.v[at, mxfp4.code_place(t, dim, 128, False)[0]] = 0
    got = _attend(s.upload())
    ref, tol = reference(s)
    assert (got[..., 96:] == 0).all()
    check(got[..., :96], ref[..., :96], tol[..., :96])


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("keys, queries", [(100, -100), (115, -118), (122, -110), (-100, 100), (-110, 118), (80, -60)])
def test_large_keys_with_small_queries(kind, keys, queries):
    """Scores of ordinary size from keys of 2^keys and queries of 2^queries, or the reverse."""
    s = Step(10, KINDS[kind], 4, 1, 64)
    for slots in s.slots:
        s.pools.scales(s.rng, slots, keys - 1, keys + 1, v=False)
    s.q = (s.q.double() * 2.0 ** queries).to(torch.bfloat16)
    s.q[:, 1] = 0
    s.scale = 2.0 ** min(3 - keys - queries, 8) / 8
    s.upload()
    check(_attend(s), *reference(s))


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("lo, hi", [(-20, 3), (-60, 3), (0, 0)])
@pytest.mark.parametrize("d", [64, 128])
def test_keys_far_apart_with_uneven_values(kind, lo, hi, d):
    """Keys whose scales are 2^lo to 2^hi, values whose first group is 2^40 above the others."""
    s = Step(11, KINDS[kind], 8, 2, d)
    for r, slots in enumerate(s.slots):
        s.pools.scales(s.rng, slots, lo, hi, v=False)
        _uneven(s, r, slice(0, None, 3))
    s.upload()
    check(_attend(s), *reference(s))
