"""What the 8-bit cache's and the rotary table's entry points refuse, before anything
reaches a GPU (nothing here launches a kernel)."""

import math

import pytest
import torch


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_36_gb300 import build
    build.build()
    import paged_kv_cache_36_gb300 as m
    return m


P = 1 << 20  # a 16-byte aligned address that is never dereferenced


@pytest.mark.parametrize("bs, hkv, d, size", [(16, 8, 128, 16512), (16, 1, 64, 1040), (16, 5, 128, 10320),
                                              (8, 8, 128, 0), (16, 0, 128, 0), (16, 8, 96, 0)])
def test_block_bytes(pkv, bs, hkv, d, size):
    assert pkv.lib().pkv_fp8_block_bytes(bs, hkv, d) == size


@pytest.mark.parametrize("name", ["pkv_reshape_and_cache_fp8", "pkv_gather_cache_fp8"])
@pytest.mark.parametrize("change, code", [
    (dict(T=0), 0), (dict(T=-1), -1), (dict(nb=0), -1), (dict(bs=32), -2), (dict(d=96), -2),
    (dict(hkv=0), -1), (dict(dtype=2), -2), (dict(rows=None), -1), (dict(slots=None), -1),
    (dict(rows=P + 8), -1), (dict(cache=P + 4), -1), (dict(ks=2 * 64 + 4), -1), (dict(ks=64), -1),
    (dict(nb=1 << 31), -2)])
def test_cache_write_and_gather(pkv, name, change, code):
    a = dict(T=3, nb=4, bs=16, hkv=2, d=64, dtype=1, rows=P, cache=P, slots=P, ks=128)
    a.update(change)
    rows, cache = [a["rows"], a["rows"]], [a["cache"], a["cache"]]
    tail = [a["T"], a["nb"], a["bs"], a["hkv"], a["d"], a["dtype"], None, None]
    if "gather" in name:
        args = cache + [a["slots"]] + rows + [a["ks"], a["ks"]] + tail
    else:
        args = rows + [a["ks"], a["ks"]] + cache + [a["slots"]] + tail
    assert getattr(pkv.lib(), name)(*args) == code


@pytest.mark.parametrize("T, code", [((1 << 20) + 1, -2), (1 << 30, -2), (1 << 20, -1)])
def test_writes_that_would_search_for_long(pkv, T, code):
    """Tokens past 2^20 are refused (and 2^20 by another check: a null table, rows off 16 bytes)."""
    tail = [T, 1 << 20, 16, 2, 64, 1, None, None]
    assert pkv.lib().pkv_rope_reshape_and_cache_fp8(P, 4 * P, 256, 6 * P, 256, 4, P, 128, 2 * P, 128, 3 * P, 3 * P, P,
                                                    None, 10, 64, 1, *tail) == code
    rows = P if code == -2 else P + 8
    assert pkv.lib().pkv_reshape_and_cache_fp8(rows, rows, 128, 128, P, P, P, *tail) == code


@pytest.mark.parametrize("change, code", [
    (dict(T=0), 0), (dict(T=-1), -1), (dict(T=1 << 31), -2), (dict(T=(1 << 30) + 1), -2), (dict(H=0), -1), (dict(rd=0), -2),
    (dict(rd=72), -2), (dict(rd=24), -2), (dict(rd=8, neox=0, dtype=1), 1), (dict(rd=8), -2),
    (dict(rd=8, dtype=0), 1), (dict(maxp=-1), -1), (dict(pos=None), -1), (dict(q=None), -1),
    (dict(qo=None), -1), (dict(table=None), -1), (dict(table=P + 8), -1), (dict(qs=64), -1),
    (dict(qos=260), -1), (dict(q=4 * P + 8), -1),
    # query_out: itself with another stride, shifted by a row, over the keys, between the queries' rows
    (dict(qo=4 * P, qos=512), -1), (dict(qo=4 * P + 512), -1), (dict(qo=P), -1), (dict(qo=2 * P + 128), -1),
    (dict(qo=4 * P + 512, qs=512, qos=512), 1), (dict(qo=4 * P + 256, qs=512, qos=512), -1)])
def test_rope(pkv, change, code):
    a = dict(T=3, nb=4, bs=16, hkv=2, H=4, d=64, dtype=1, pos=P, q=4 * P, qs=256, qo=6 * P, qos=256,
             table=P, maxp=10, rd=64, neox=1)
    a.update(change)
    if code == 1:   # allowed: shown by the refusal of a later check only
        a["qo"], code = (a["qo"] if "qo" in change else None), -1
        if "qo" in change:
            a["q"], a["qo"] = a["q"] + 8, a["qo"] + 8    # both off their alignment, still apart
    rc = pkv.lib().pkv_rope_reshape_and_cache_fp8(
        a["pos"], a["q"], a["qs"], a["qo"], a["qos"], a["H"], P, 128, 2 * P, 128, 3 * P, 3 * P, P, a["table"],
        a["maxp"], a["rd"], a["neox"], a["T"], a["nb"], a["bs"], a["hkv"], a["d"], a["dtype"], None, None)
    assert rc == code


@pytest.mark.parametrize("change, code", [
    (dict(T=0), 0), (dict(R=0), 0), (dict(T=-1), -1), (dict(T=(1 << 30) + 1), -2), (dict(R=9000), -2), (dict(bs=8), -2),
    (dict(d=80), -2), (dict(H=5), -1), (dict(H=34, hkv=2), -2), (dict(ws=None), -3),
    (dict(wsb=16), -3), (dict(q=None), -1), (dict(bt=None), -1), (dict(q=P + 2), -1),
    (dict(qs=4 * 64 + 4), -1), (dict(qs=64), -1), (dict(width=0), -1), (dict(width=9), -1),
    (dict(mql=-1), -1), (dict(nb=0), -1), (dict(scale=math.nan), -1), (dict(scale=math.inf), -1),
    (dict(scale=3e38), -1),
    # 4096 requests that might share 2^19 rows of 8 KV heads: 2^31 tiles of 8 tokens
    (dict(R=4096, T=1 << 19, H=128, hkv=8, qs=8192), -2)])
def test_attention(pkv, change, code):
    a = dict(T=3, R=2, nb=4, bs=16, H=4, hkv=2, d=64, q=P, bt=P, ws=P, wsb=1 << 40, qs=256, width=8,
             stride=8, mql=0, scale=0.125)
    a.update(change)
    rc = pkv.lib().pkv_paged_attention_varlen_fp8(
        a["q"], a["qs"], P, P, a["bt"], a["stride"], a["width"], P, P, P, a["scale"], P, a["qs"], a["T"],
        a["R"], a["nb"], a["bs"], a["H"], a["hkv"], a["d"], a["mql"], a["ws"], a["wsb"], None)
    assert rc == code
    if code:
        assert b"pkv_paged_attention_varlen_fp8" in pkv.lib().pkv_last_error()

@pytest.mark.parametrize("R, width", [(1, 0x7fffffff - 1), (1, 0x7fffffff - 15), (2, 1 << 30), (8192, 1 << 18)])
def test_block_tables_that_32_bits_do_not_count(pkv, R, width):
    """With what a request and a rounded division add to their entries."""
    assert pkv.lib().pkv_paged_attention_varlen_fp8(
        P, 256, P, P, P, width, width, P, P, P, 0.125, P, 256, 3, R, 4, 16, 4, 2, 64, 1, P, 1 << 40, None) == -2


@pytest.mark.parametrize("H, hkv, d", [(4, 3, 64), (34, 2, 64), (0, 1, 64), (8, 8, 96)])
def test_workspace_of_unsupported_heads(pkv, H, hkv, d):
    assert pkv.lib().pkv_fp8_attention_workspace_bytes(H, hkv, d) == 0
    with pytest.raises(ValueError):
        pkv.new_workspace_fp8(H, hkv, d, device="cpu")


@pytest.mark.parametrize("change, code", [
    (dict(n=0), 0), (dict(n=-1), -1), (dict(start=-1), -1), (dict(rd=0), -1), (dict(rd=7), -1),
    (dict(rd=514), -2), (dict(n=1 << 27), -2), (dict(start=1 << 26), -2), (dict(base=1.0), -1),
    (dict(base=math.nan), -1), (dict(base=math.inf), -1), (dict(scaling=5), -1), (dict(scaling=-1), -1),
    (dict(scaling=1, factor=0.5), -1), (dict(scaling=1, factor=math.inf), -1), (dict(scaling=2, rd=2), -1),
    (dict(scaling=3, length=0), -1), (dict(scaling=4, low=0.0), -1), (dict(scaling=3, low=32.0), -1),
    (dict(scaling=3, high=math.inf), -1), (dict(att=math.nan), -1), (dict(out=None), -1), (dict(out=P + 4), -1)])
def test_table(pkv, change, code):
    a = dict(out=P, n=4, start=0, rd=8, base=1e4, scaling=0, factor=2.0, length=100, low=1.0, high=32.0, att=1.0)
    a.update(change)
    assert pkv.lib().pkv_build_cos_sin_cache(
        a["out"], a["n"], a["start"], a["rd"], a["base"], a["scaling"], a["factor"], a["length"], a["low"],
        a["high"], a["att"], None) == code
    if code:
        assert b"pkv_build_cos_sin_cache" in pkv.lib().pkv_last_error()


@pytest.mark.parametrize("factor", [3.5e38, -1e300])
def test_table_with_a_factor_past_float32(pkv, factor):
    assert pkv.lib().pkv_build_cos_sin_cache(P, 4, 0, 8, 1e4, 0, 2.0, 100, 1.0, 32.0, factor, None) == -1


def test_python_argument_checks(pkv):
    bf, u8, i64, i32 = torch.bfloat16, torch.uint8, torch.int64, torch.int32
    k = torch.zeros(3, 2, 64, dtype=bf)
    kc, vc = pkv.new_cache_fp8(4, 2, 64, device="cpu")
    assert kc.shape == (4, 2080) and kc.dtype == u8
    slots = torch.zeros(3, dtype=i64)
    with pytest.raises(ValueError, match="CUDA device"):
        pkv.reshape_and_cache_fp8(k, k, kc, vc, slots)
    with pytest.raises(ValueError, match="key_cache"):
        pkv.reshape_and_cache_fp8(torch.zeros(3, 4, 64, dtype=bf), torch.zeros(3, 4, 64, dtype=bf), kc, vc, slots)
    with pytest.raises(TypeError, match="slot_mapping"):
        pkv.reshape_and_cache_fp8(k, k, kc, vc, slots.to(i32))
    with pytest.raises(ValueError, match="slot_mapping"):
        pkv.gather_cache_fp8(kc, vc, slots[:2], k, k)
    with pytest.raises(ValueError, match="one shape"):
        pkv.gather_cache_fp8(kc, vc, slots, k, k.float())
    with pytest.raises(TypeError):
        pkv.gather_cache_fp8(kc.view(torch.int8), vc, slots, k, k)
    with pytest.raises(ValueError):
        pkv.fp8_block_bytes(8, 96)
    # a 4-bit cache is not an 8-bit one
    mk, mv = pkv.new_cache_mxfp4(4, 2, 64, device="cpu")
    with pytest.raises(ValueError, match="key_cache"):
        pkv.gather_cache_fp8(mk, mv, slots, k, k)

    rope = pkv.rope_reshape_and_cache_fp8
    q, table = torch.zeros(3, 4, 64, dtype=bf), torch.zeros(9, 64)
    with pytest.raises(ValueError, match="query"):
        rope(slots, q.float(), k, k, kc, vc, slots, table)
    with pytest.raises(ValueError, match="query_out"):
        rope(slots, q, k, k, kc, vc, slots, table, query_out=q[:, :2])
    with pytest.raises(TypeError, match="positions"):
        rope(slots.to(i32), q, k, k, kc, vc, slots, table)
    with pytest.raises(TypeError, match="cos_sin_cache"):
        rope(slots, q, k, k, kc, vc, slots, table.double())
    with pytest.raises(ValueError, match="CUDA device"):
        rope(slots, q, k, k, kc, vc, slots, table)

    q = torch.zeros(2, 4, 64, dtype=bf)
    bt = torch.zeros(2, 2, dtype=i32)
    qsl, seq, past = (torch.tensor(x, dtype=i32) for x in ([0, 1, 2], [1, 1], [0, 0]))
    attend = pkv.paged_attention_varlen_fp8
    with pytest.raises(TypeError, match="bfloat16"):
        attend(q.float(), kc, vc, bt, qsl, seq, past, 1.0)
    with pytest.raises(TypeError, match="seq_lens"):
        attend(q, kc, vc, bt, qsl, seq.long(), past, 1.0)
    with pytest.raises(ValueError, match="query_start_loc"):
        attend(q, kc, vc, bt, qsl[:2], seq, past, 1.0)
    with pytest.raises(ValueError, match="block_table"):
        attend(q, kc, vc, bt[:1], qsl, seq, past, 1.0)
    with pytest.raises(ValueError, match="key_cache"):
        attend(q, kc[:, :1000].contiguous(), vc, bt, qsl, seq, past, 1.0)

    with pytest.raises(ValueError, match="scaling"):
        pkv.build_cos_sin_cache(4, 8, scaling="cubic")
    with pytest.raises(ValueError, match="CUDA device"):
        pkv.build_cos_sin_cache(4, 8, device="cpu")
    with pytest.raises(ValueError, match="CUDA device"):
        pkv.build_cos_sin_cache(4, 8, out=torch.zeros(4, 8))
    with pytest.raises(ValueError, match="shape"):
        pkv.build_cos_sin_cache(4, 8, out=torch.zeros(4, 9))
    with pytest.raises(TypeError, match="out"):
        pkv.build_cos_sin_cache(4, 8, out=torch.zeros(4, 8).double())
