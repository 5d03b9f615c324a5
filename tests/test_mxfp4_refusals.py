"""What the 4-bit cache's and the device metadata's entry points refuse, before
anything reaches a GPU (nothing here launches a kernel)."""

import pytest
import torch


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_36_gb300 import build
    build.build()
    import paged_kv_cache_36_gb300 as m
    return m


P = 1 << 20  # a 16-byte aligned address that is never dereferenced


@pytest.mark.parametrize("bs, hkv, d, size", [(16, 8, 128, 8704), (16, 1, 64, 544), (16, 5, 128, 5440),
                                              (8, 8, 128, 0), (16, 0, 128, 0), (16, 8, 96, 0)])
def test_block_bytes(pkv, bs, hkv, d, size):
    assert pkv.lib().pkv_mxfp4_block_bytes(bs, hkv, d) == size


@pytest.mark.parametrize("name", ["pkv_reshape_and_cache_mxfp4", "pkv_gather_cache_mxfp4"])
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


@pytest.mark.parametrize("change, code", [
    (dict(T=0), 0), (dict(R=0), 0), (dict(T=-1), -1), (dict(R=9000), -2), (dict(bs=8), -2),
    (dict(d=80), -2), (dict(H=5), -1), (dict(H=34, hkv=2), -2), (dict(ws=None), -3),
    (dict(wsb=16), -3), (dict(q=None), -1), (dict(bt=None), -1), (dict(q=P + 2), -1),
    (dict(qs=4 * 64 + 4), -1), (dict(qs=64), -1), (dict(width=0), -1), (dict(width=9), -1),
    (dict(mql=-1), -1), (dict(nb=0), -1)])
def test_attention(pkv, change, code):
    a = dict(T=3, R=2, nb=4, bs=16, H=4, hkv=2, d=64, q=P, bt=P, ws=P, wsb=1 << 40, qs=256, width=8,
             stride=8, mql=0)
    a.update(change)
    rc = pkv.lib().pkv_paged_attention_varlen_mxfp4(
        a["q"], a["qs"], P, P, a["bt"], a["stride"], a["width"], P, P, P, 0.125, P, a["qs"], a["T"],
        a["R"], a["nb"], a["bs"], a["H"], a["hkv"], a["d"], a["mql"], a["ws"], a["wsb"], None)
    assert rc == code
    if code:
        assert b"pkv_paged_attention_varlen_mxfp4" in pkv.lib().pkv_last_error()

@pytest.mark.parametrize("R, width", [(1, 0x7fffffff - 1), (1, 0x7fffffff - 15), (2, 1 << 30), (8192, 1 << 18)])
def test_block_tables_that_32_bits_do_not_count(pkv, R, width):
    """With what a request and a rounded division add to their entries."""
    assert pkv.lib().pkv_paged_attention_varlen_mxfp4(
        P, 256, P, P, P, width, width, P, P, P, 0.125, P, 256, 3, R, 4, 16, 4, 2, 64, 1, P, 1 << 40, None) == -2


@pytest.mark.parametrize("H, hkv, d", [(4, 3, 64), (34, 2, 64), (0, 1, 64), (8, 8, 96)])
def test_workspace_of_unsupported_heads(pkv, H, hkv, d):
    assert pkv.lib().pkv_mxfp4_attention_workspace_bytes(H, hkv, d) == 0
    with pytest.raises(ValueError):
        pkv.new_workspace_mxfp4(H, hkv, d, device="cpu")


def _tables(pkv, **change):
    # distinct, well separated addresses
    names = ["new", "held", "table", "ring", "state", "out", "qsl", "seq", "slots", "pos"]
    a = {n: P * (i + 1) for i, n in enumerate(names)}
    a.update(R=4, width=8, stride=8, size=64, bs=16, T=100)
    a.update(change)
    return pkv.lib().pkv_build_step_metadata(
        a["new"], a["held"], a["R"], a["table"], a["stride"], a["width"], a["ring"], a["size"],
        a["state"], a["out"], a["bs"], a["T"], a["qsl"], a["seq"], a["slots"], a["pos"], None, None)


@pytest.mark.parametrize("change, code", [
    (dict(R=-1), -1), (dict(T=-1), -1), (dict(size=-1), -1), (dict(width=-1), -1), (dict(bs=8), -2),
    (dict(R=8193), -2), (dict(T=1 << 31), -2), (dict(stride=4), -1), (dict(new=None), -1),
    (dict(held=None), -1), (dict(table=None), -1), (dict(ring=None), -1), (dict(state=None), -1),
    (dict(out=None), -1), (dict(qsl=None), -1), (dict(seq=None), -1), (dict(slots=None), -1),
    # lengths advanced in place, a slot map over the table, a ring's state over another's
    (dict(seq=2 * P), -1), (dict(slots=3 * P + 64), -1), (dict(out=5 * P + 8), -1),
    (dict(pos=9 * P + 8), -1), (dict(qsl=4 * P), -1)])
def test_step_metadata(pkv, change, code):
    assert _tables(pkv, **change) == code
    assert b"pkv_build_step_metadata" in pkv.lib().pkv_last_error()


def test_python_argument_checks(pkv):
    bf, u8, i64, i32 = torch.bfloat16, torch.uint8, torch.int64, torch.int32
    k = torch.zeros(3, 2, 64, dtype=bf)
    kc, vc = pkv.new_cache_mxfp4(4, 2, 64, device="cpu")
    assert kc.shape == (4, 1088) and kc.dtype == u8
    slots = torch.zeros(3, dtype=i64)
    with pytest.raises(ValueError, match="CUDA device"):
        pkv.reshape_and_cache_mxfp4(k, k, kc, vc, slots)
    with pytest.raises(ValueError, match="key_cache"):
        pkv.reshape_and_cache_mxfp4(torch.zeros(3, 4, 64, dtype=bf), torch.zeros(3, 4, 64, dtype=bf),
                                    kc, vc, slots)
    with pytest.raises(TypeError, match="slot_mapping"):
        pkv.reshape_and_cache_mxfp4(k, k, kc, vc, slots.to(i32))
    with pytest.raises(ValueError, match="slot_mapping"):
        pkv.gather_cache_mxfp4(kc, vc, slots[:2], k, k)
    with pytest.raises(ValueError, match="one shape"):
        pkv.gather_cache_mxfp4(kc, vc, slots, k, k.float())
    with pytest.raises(TypeError):
        pkv.gather_cache_mxfp4(kc.view(torch.int8), vc, slots, k, k)
    with pytest.raises(ValueError, match="contiguous"):
        pkv.gather_cache_mxfp4(torch.zeros(4, 2176, dtype=u8)[:, :1088], vc, slots, k, k)
    with pytest.raises(ValueError):
        pkv.mxfp4_block_bytes(8, 96)

    q = torch.zeros(2, 4, 64, dtype=bf)
    bt = torch.zeros(2, 2, dtype=i32)
    qsl, seq, past = (torch.tensor(x, dtype=i32) for x in ([0, 1, 2], [1, 1], [0, 0]))
    attend = pkv.paged_attention_varlen_mxfp4
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

    build = pkv.build_step_metadata
    ring, state = torch.zeros(8, dtype=i32), torch.zeros(4, dtype=i64)
    with pytest.raises(TypeError, match="query_lens"):
        build(seq.long(), past, bt, ring, state, 4)
    with pytest.raises(ValueError, match="free_state"):
        build(seq, past, bt, ring, state[:3], 4)
    with pytest.raises(ValueError, match="block_table"):
        build(seq, past, bt[:1], ring, state, 4)
    with pytest.raises(ValueError, match="CUDA device"):
        build(seq, past, bt, ring, state, 4)
