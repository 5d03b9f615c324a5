"""Offsets of query rows that are garbage: refused by the kernels' own checks."""

import pytest
import torch

from tests.mxfp4_support import Step, check

pytestmark = pytest.mark.gpu

TOP, LOW = 2 ** 31 - 1, -2 ** 31


@pytest.mark.parametrize("pair", [(TOP, LOW), (TOP, LOW + 7), (4, 5), (4, 9), (-1, 0), (-3, 4), (LOW, TOP)])
@pytest.mark.parametrize("longest", [0, 1])
def test_offsets_outside_the_batch(pair, longest):
    """A request's rows are [first, second) of four tokens, one or several as int32 counts them.
    Where they are rows at all, they are left alone and the call says so."""
    import paged_kv_cache_36_gb300 as pkv
    s = Step(1, [(1, 30), (1, 90), (2, 60)], 8, 2, 64).upload()
    n = (pair[1] - pair[0] + 2 ** 31) % 2 ** 32 - 2 ** 31
    qsl = torch.tensor([pair[0], pair[1]], dtype=torch.int32, device="cuda")
    past = s.dpast[:1]
    ws = pkv.new_workspace_mxfp4(8, 2, 64)
    out = torch.full_like(s.dq, 3.0)
    pkv.paged_attention_varlen_mxfp4(s.dq, s.kc, s.vc, s.bt[:1], qsl, past + n, past, s.scale, out=out,
                                     workspace=ws, max_query_len=longest)
    rows = n == 1 or (n > 1 and longest != 1)
    assert pkv.read_error_word(ws) == (pkv.ERR_METADATA if rows else 0)
    assert (out == 3.0).all()
    # and the workspace is as good as before
    ws[:4] = 0
    check(pkv.paged_attention_varlen_mxfp4(*s.args(), workspace=ws), *s.reference())
