"""Values of a context further apart than float32's exponent range, within a bound that goes by
what each row sees and by weight times value (tests/mxfp4_bounds.py)."""

import numpy as np
import pytest

from oracle import mxfp4
from tests.mxfp4_bounds import check, reference
from tests.mxfp4_support import Step

pytestmark = pytest.mark.gpu

REQS = [[(1, 700), (1, 40)], [(20, 270)], [(60, 900)]]   # decode, prefill, converted ahead


def _attend(s):
    import paged_kv_cache_36_gb300 as pkv
    ws = pkv.new_workspace_mxfp4(s.H, s.hkv, s.d)
    got = pkv.paged_attention_varlen_mxfp4(*s.args(), workspace=ws, max_query_len=max(s.q_len))
    assert pkv.read_error_word(ws) == 0
    return got


@pytest.mark.parametrize("reqs", REQS)
@pytest.mark.parametrize("first, then", [(-110, 60), (60, -110), (-70, 70), (100, 100), (-120, -120), (0, 12), (12, 0)])
@pytest.mark.parametrize("part", [0.25, 0.97])
def test_values_of_two_kinds(reqs, first, then, part):
    """V scales 2^first, and 2^then from some position on: rows before it keep their precision."""
    s = Step(91, reqs, 16, 1, 64)
    for slots in s.slots:
        n = int(part * len(slots))
        s.pools.scales(s.rng, slots[:n], first, first, k=False)
        s.pools.scales(s.rng, slots[n:], then, then, k=False)
    s.upload()
    check(_attend(s), *reference(s), tight=0.6)


@pytest.mark.parametrize("reqs", REQS)
@pytest.mark.parametrize("lo, hi", [(-110, 100), (-126, 60), (-40, 12), (-60, 40), (-12, 12), (-5, 6)])
@pytest.mark.parametrize("d", [64, 128])
def test_values_of_every_kind(reqs, lo, hi, d):
    s = Step(92, reqs, 16, 1, d)
    s.pools.scales(s.rng, np.concatenate(s.slots), lo, hi, k=False)
    s.upload()
    check(_attend(s), *reference(s), tight=0.6)


@pytest.mark.parametrize("reqs", REQS)
@pytest.mark.parametrize("low, large", [(96, 60), (96, 95), (96, -60), (32, 30)])
def test_scores_and_values_far_apart(reqs, low, large):
    """A third of the keys are 2^-low as likely as the others, with values 2^large times
    theirs."""
    s = Step(93, reqs, 16, 1, 64)
    s.q[:, :, :] = 0
    s.q[:, :, 0] = 1.0
    s.scale = float(np.log(2.0))
    for r, slots in enumerate(s.slots):
        least = np.array([(j * 7 + r) % 3 == 0 for j in range(len(slots))])
        for j, slot in enumerate(slots.tolist()):
            row = np.zeros((1, 64))
            row[0, 0] = -low if least[j] else 0.25 * (j % 3)
            mxfp4.write_row(s.pools.k, slot, row, True)
        s.pools.scales(s.rng, slots[least], large // 2, large // 2, k=False)
        s.pools.scales(s.rng, slots[~least], large // 2 - large, large // 2 - large, k=False)
    s.upload()
    check(_attend(s), *reference(s))
