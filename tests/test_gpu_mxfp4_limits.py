"""The 4-bit attention at the ends of its ranges: the most requests, more KV heads
than a CTA has warps, queries that are NaN, and the error word checked by the call."""

import numpy as np
import pytest
import torch

from tests.mxfp4_support import Step, check

pytestmark = pytest.mark.gpu


def _pkv():
    import paged_kv_cache_36_gb300 as pkv
    return pkv


@pytest.mark.parametrize("reqs, heads, hkv, d", [
    ([(1, 70), (1, 0), (1, 333)], 40, 20, 64),               # two passes over the heads
    ([(1, 70), (1, 500)], 144, 9, 128),                      # 16 query heads of 9
    ([(1, 200), (40, 17), (1, 3)], 33, 33, 64),
    ([(70, 900), (1, 100)], 144, 9, 64),                     # converted ahead
])
def test_many_kv_heads(reqs, heads, hkv, d):
    pkv = _pkv()
    s = Step(heads + d, reqs, heads, hkv, d).upload()
    ws = pkv.new_workspace_mxfp4(heads, hkv, d)
    got = pkv.paged_attention_varlen_mxfp4(*s.args(), workspace=ws)
    assert pkv.read_error_word(ws) == 0
    check(got, *s.reference())


@pytest.mark.parametrize("n", [30, 45, 90])
def test_joins_of_every_width(n):
    """960, 1440 and 2880 query heads of 128 in a step: their ranges are joined by 8, 16 and
    32 lanes."""
    pkv = _pkv()
    rng = np.random.default_rng(n)
    s = Step(70 + n, [(1, int(p)) for p in rng.integers(0, 400, n)] + [(1, 3000)], 32, 8, 128).upload()
    ws = pkv.new_workspace_mxfp4(32, 8, 128)
    got = pkv.paged_attention_varlen_mxfp4(*s.args(), workspace=ws, max_query_len=1)
    assert pkv.read_error_word(ws) == 0
    check(got, *s.reference())


def test_the_most_requests():
    """8192 requests: decode rows, short chunks, and a few that are converted ahead."""
    pkv = _pkv()
    rng = np.random.default_rng(3)
    reqs = [(1, int(p)) for p in rng.integers(0, 40, 8192)]
    for r in rng.choice(8192, 900, replace=False):
        reqs[r] = (int(rng.integers(0, 4)), int(rng.integers(0, 50)))
    for r in (0, 4095, 4096, 8191):
        reqs[r] = (230 + r % 7, 800)
    s = Step(4, reqs, 4, 1, 64).upload()
    ws = pkv.new_workspace_mxfp4(4, 1, 64)
    got = pkv.paged_attention_varlen_mxfp4(*s.args(), workspace=ws)
    assert pkv.read_error_word(ws) == 0
    check(got, *s.reference())


@pytest.mark.parametrize("reqs", [[(1, 90), (1, 300)], [(20, 70)], [(60, 870)]])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_query_that_is_not_finite_spoils_its_own_row(reqs, value):
    pkv = _pkv()
    s = Step(61, reqs, 16, 1, 64).upload()
    ref, tol = s.reference()
    s.dq[0, 3, 17] = value
    got = pkv.paged_attention_varlen_mxfp4(*s.args(), max_query_len=max(s.q_len)).cpu()
    keep = torch.ones(s.T, 16, dtype=torch.bool)
    keep[0, 3] = False
    assert torch.isnan(got[0, 3]).all()
    check(got, ref, tol, rows=keep)


def test_the_call_checks_the_error_word_on_request(monkeypatch):
    pkv = _pkv()
    s = Step(62, [(1, 90), (60, 30)], 16, 1, 64)
    s.table[1, 1] = 10 ** 6
    s.upload()
    monkeypatch.setenv("PKV_VALIDATE", "1")
    with pytest.raises(pkv.PkvError):
        pkv.paged_attention_varlen_mxfp4(*s.args())
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    k = torch.ones(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    far = torch.tensor([1 << 40], device="cuda")
    with pytest.raises(pkv.PkvError):
        pkv.reshape_and_cache_mxfp4(k, k, s.kc, s.vc, far, error_word=err)
