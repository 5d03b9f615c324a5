"""GPU tests of the 4-bit prefill over key tiles that are converted ahead (requests
of at least 4 query tiles of 128 / G tokens and 8 key tiles of 128), within the bound
of tests/mxfp4_support.py: its arithmetic is the direct kernel's, with bases of 128
keys instead of 32."""

import numpy as np
import pytest
import torch

from oracle import mxfp4
from tests.mxfp4_support import Step, check

pytestmark = pytest.mark.gpu

IMAGE_ROOM = 256 << 20


def _pkv():
    import paged_kv_cache_36_gb300 as pkv
    return pkv


def _attend(s, **kw):
    pkv = _pkv()
    ws = pkv.new_workspace_mxfp4(s.H, s.hkv, s.d)
    got = pkv.paged_attention_varlen_mxfp4(*s.args(), workspace=ws, max_query_len=max(s.q_len), **kw)
    assert pkv.read_error_word(ws) == 0
    return got


@pytest.mark.parametrize("reqs, heads, hkv, d", [
    # 16 query heads a KV head: 8 tokens a query tile, images from 25 tokens and 897 keys on
    ([(25, 872)], 16, 1, 64),
    ([(57, 967)], 16, 1, 128),                    # ends with a key tile
    ([(64, 961)], 32, 2, 128),                    # one key into the next
    ([(24, 1300), (25, 1300)], 16, 1, 64),        # one on each side of the rule
    ([(30, 866), (30, 867)], 16, 1, 128),         # and of the other
    ([(1, 40), (70, 900), (0, 3), (9, 100), (920, 0), (1, 500), (2, 2)], 32, 2, 64),
    ([(90, 1900), (30, 0), (130, 901)], 16, 1, 128),
    ([(230, 710)], 12, 3, 128),                   # 4 a KV head
    ([(160, 933)], 28, 4, 64),                    # 7, tiles of 18 tokens
    ([(1000, 24)], 2, 2, 64),                     # one: 128 tokens a tile
])
def test_attention(reqs, heads, hkv, d):
    s = Step(len(reqs) * 77 + heads + d, reqs, heads, hkv, d, stride_pad=1, table_pad=2).upload()
    check(_attend(s), *s.reference())


@pytest.mark.parametrize("lo, hi", [(-40, 12), (-126, -100), (-60, 40), (-7, 7), (20, 21)])
@pytest.mark.parametrize("what", ["keys", "values"])
def test_scales_over_many_binades(lo, hi, what):
    if what == "keys" and hi > 12:
        lo, hi = lo // 8, hi // 8   # scores a softmax can tell apart
    s = Step(hi - lo, [(57, 860)], 16, 1, 128)
    s.pools.scales(s.rng, np.concatenate(s.slots), lo, hi, k=what == "keys", v=what == "values")
    s.upload()
    check(_attend(s), *s.reference())


@pytest.mark.parametrize("is_key", [True, False])
@pytest.mark.parametrize("tok", [3, 895, 896, 930])
def test_a_nan_group_stays_with_its_rows(is_key, tok):
    """Past, at and behind the new tokens; in the first and the second key tile."""
    s = Step(17 + tok, [(60, 880)], 16, 1, 128)
    slot = int(s.slots[0][tok])
    pool = s.pools.k if is_key else s.pools.v
    pool[slot // 16, mxfp4.scale_place(slot % 16, 1, 128, is_key)] = 255
    for dim in range(32, 64):
        byte, _ = mxfp4.code_place(slot % 16, dim, 128, is_key)
        pool[slot // 16, byte] = 0
    s.nan = (0,)
    got = _attend(s.upload()).double().cpu()
    ref, tol = s.reference()
    bad = torch.zeros_like(ref, dtype=torch.bool)
    bad[max(0, tok - 880):, :, (slice(None) if is_key else slice(32, 64))] = True
    assert torch.isnan(ref[bad]).all() and torch.isfinite(ref[~bad]).all()
    assert torch.isnan(got[bad]).all()
    check(got, ref, tol, rows=~bad)


def test_an_outlier_that_no_row_but_the_last_sees():
    """The last token's K and V are 2^60 times the others': the rows before it
    keep their precision."""
    n = 60
    s = Step(23, [(n, 900)], 16, 1, 64)
    plain_ref, plain_tol = s.reference()
    s.pools.scales(s.rng, s.slots[0][-1:], 60, 60)
    got = _attend(s.upload())
    check(got, plain_ref, plain_tol, rows=slice(0, n - 1))


def test_bad_blocks_and_bad_metadata():
    pkv = _pkv()
    reqs = [(60, 900), (58, 870), (1, 33)]
    ref, tol = Step(8, reqs, 16, 1, 64).reference()
    for col, bad in ((2, -1), (15, 10 ** 6)):
        t = Step(8, reqs, 16, 1, 64)
        t.table[0, col] = bad
        t.upload()
        ws = pkv.new_workspace_mxfp4(16, 1, 64)
        got = pkv.paged_attention_varlen_mxfp4(*t.args(), workspace=ws)
        assert pkv.read_error_word(ws) == pkv.ERR_BLOCK_ID
        zero = Step(8, reqs, 16, 1, 64)   # reads as zeros
        blk = int(zero.table[0, col])
        zero.pools.k[blk] = 0
        zero.pools.v[blk] = 0
        check(got, *zero.reference())
    for r, field, bad in ((0, "dseq", 959), (1, "dpast", -1), (0, "dseq", 10 ** 9)):
        t = Step(8, reqs, 16, 1, 64).upload()
        getattr(t, field)[r] = bad
        if field == "dpast":
            t.dseq[r] = bad + t.q_len[r]
        ws = pkv.new_workspace_mxfp4(16, 1, 64)
        out = torch.full_like(t.dq, 3.0)
        got = pkv.paged_attention_varlen_mxfp4(*t.args(), out=out, workspace=ws)
        assert pkv.read_error_word(ws) == pkv.ERR_METADATA
        keep = torch.ones(t.T, dtype=torch.bool)
        keep[int(t.qsl[r]):int(t.qsl[r + 1])] = False
        check(got, ref, tol, rows=keep)
        assert (got.cpu()[~keep] == 3.0).all()


@pytest.mark.parametrize("tiles", [0, 7, 8, 9, 16, 17, 25])
def test_workspaces_with_less_room(tiles):
    """Key tiles 9, 8 and 8: the requests that find no room are computed directly."""
    pkv = _pkv()
    s = Step(41, [(60, 1000), (57, 900), (80, 900), (1, 9)], 16, 1, 128).upload()
    full = pkv.mxfp4_attention_workspace_bytes(16, 1, 128)
    image = 2 * 32768 + 1152       # K, V, scales
    least = full - IMAGE_ROOM // image * image
    ws = torch.full((least + tiles * image + 64,), 255, dtype=torch.uint8, device="cuda")
    ws[:256] = 0
    out = torch.zeros_like(s.dq)
    got = pkv.paged_attention_varlen_mxfp4(*s.args(), out=out, workspace=ws[:least + tiles * image])
    assert pkv.read_error_word(ws) == 0
    check(got, *s.reference())
    assert (ws[-64:] == 255).all()
    with pytest.raises(pkv.PkvError):
        pkv.paged_attention_varlen_mxfp4(*s.args(), workspace=ws[:least - 16])


def test_two_graphs_that_share_a_workspace():
    pkv = _pkv()
    ws = pkv.new_workspace_mxfp4(16, 1, 64)
    steps = [Step(51, [(60, 870), (1, 300)], 16, 1, 64).upload(),
             Step(52, [(1, 20), (99, 840), (3, 5)], 16, 1, 64).upload()]
    graphs, outs = [], []
    for s in steps:
        out = torch.zeros_like(s.dq)
        pkv.paged_attention_varlen_mxfp4(*s.args(), workspace=ws, out=out)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pkv.paged_attention_varlen_mxfp4(*s.args(), workspace=ws, out=out)
        graphs.append(g)
        outs.append(out)
    want = [s.reference() for s in steps]
    for i in (0, 1, 1, 0):
        outs[i].zero_()
        graphs[i].replay()
        check(outs[i], *want[i])
    assert pkv.read_error_word(ws) == 0
