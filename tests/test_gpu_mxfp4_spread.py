"""The 4-bit attention where values next to each other are further apart than float32's
exponent range: within the bound of tests/mxfp4_support.py, which goes by the values a row
sees."""

import numpy as np
import pytest
import torch

from oracle import mxfp4
from tests.mxfp4_support import Step, check

pytestmark = pytest.mark.gpu

REQS = [[(1, 700), (1, 40)], [(20, 270)], [(60, 900)]]   # decode, prefill, converted ahead


def _attend(s):
    import paged_kv_cache_36_gb300 as pkv
    ws = pkv.new_workspace_mxfp4(s.H, s.hkv, s.d)
    got = pkv.paged_attention_varlen_mxfp4(*s.args(), workspace=ws, max_query_len=max(s.q_len))
    assert pkv.read_error_word(ws) == 0
    return got


@pytest.mark.parametrize("reqs", REQS)
@pytest.mark.parametrize("first, then", [(-110, 60), (60, -110), (-70, 70), (100, 100), (-120, -120)])
@pytest.mark.parametrize("part", [0.25, 0.97])
def test_values_of_two_kinds(reqs, first, then, part):
    """V scales 2^first, and 2^then from some position on."""
    s = Step(81, reqs, 16, 1, 64)
    for slots in s.slots:
        n = int(part * len(slots))
        s.pools.scales(s.rng, slots[:n], first, first, k=False)
        s.pools.scales(s.rng, slots[n:], then, then, k=False)
    s.upload()
    check(_attend(s), *s.reference())


@pytest.mark.parametrize("reqs", REQS)
@pytest.mark.parametrize("lo, hi", [(-110, 100), (-126, 60)])
def test_values_of_every_kind(reqs, lo, hi):
    s = Step(82, reqs, 16, 1, 128)
    s.pools.scales(s.rng, np.concatenate(s.slots), lo, hi, k=False)
    s.upload()
    check(_attend(s), *s.reference())


@pytest.mark.parametrize("reqs", REQS)
@pytest.mark.parametrize("big", [0, 1])
def test_scores_and_values_far_apart(reqs, big):
    """Half of the keys have scores some 100 octaves below the others', and values 100 octaves
    above (or below) theirs."""
    s = Step(83, reqs, 16, 1, 64)
    s.q[:, :, :] = 0
    s.q[:, :, 0] = 16.0
    s.scale = 1.0
    for r, slots in enumerate(s.slots):
        for j, slot in enumerate(slots.tolist()):
            low = (j * 7 + r) % 3 == 0
            row = np.zeros(64)
            row[0] = -4.0 if low else 0.25 * (j % 3)
            mxfp4.write_row(s.pools.k, slot, row[None], True)
        low = np.array([(j * 7 + r) % 3 == 0 for j in range(len(slots))])
        s.pools.scales(s.rng, slots[low], 60 if big else -60, 60 if big else -60, k=False)
        s.pools.scales(s.rng, slots[~low], -40 if big else 40, -40 if big else 40, k=False)
    s.upload()
    check(_attend(s), *s.reference())


@pytest.mark.parametrize("reqs", REQS)
def test_scores_of_a_million(reqs):
    """One key takes all of a row's weight, wherever it is: its value is the result."""
    s = Step(84, reqs, 16, 1, 64, lo=14, hi=16)
    s.pools.scales(s.rng, np.concatenate(s.slots), -3, 2, k=False)
    s.upload()
    ref, tol = s.reference()
    got = _attend(s)
    check(got, ref, tol)
    # rows whose first two scores are 64 apart or more have one weight that counts
    one = torch.ones(s.T, s.H, dtype=torch.bool)
    for r in range(s.R):
        k, _ = s.history(r)
        for i in range(s.q_len[r]):
            t, n = int(s.qsl[r]) + i, s.past[r] + i + 1
            top = (s.q[t].double() @ k[:n, 0].T * s.scale).topk(min(2, n), 1).values
            one[t] = top[:, 0] - top[:, -1] > 64.0
    assert one.float().mean() > 0.9
    # (the others' weights are e^-64 = 1.6e-28 at most, 960 keys of values up to 24: below
    # 1e-20 together, which is all there is where that one's value is zero)
    assert ((got.cpu().double() - ref).abs()[one] <= 2.0 ** -6 * ref.abs()[one] + 1e-20).all()
