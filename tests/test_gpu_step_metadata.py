"""The device-built step metadata against the oracle and the host scheduler, and
whole serving steps on it: tables, RoPE, 4-bit cache write, attention."""

import numpy as np
import pytest
import torch

from oracle import attention as oa
from oracle import mxfp4

pytestmark = pytest.mark.gpu

I32, I64 = torch.int32, torch.int64


def _pkv():
    import paged_kv_cache_36_gb300 as pkv
    return pkv


def _dev(x, dtype=I32):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


def _case(rng, reqs, new_hi, held_hi, width, spare=3, wrap=True):
    held = rng.integers(0, held_hi + 1, reqs)
    new = rng.integers(0, new_hi + 1, reqs)
    have = -(-held // 16)
    need = -(-(held + new) // 16) - have
    ids = rng.permutation(int(have.sum() + need.sum()) + spare)
    table = np.full((reqs, width), -1, np.int64)
    at = 0
    for r in range(reqs):
        table[r, :have[r]] = ids[at:at + have[r]]
        at += have[r]
    free = ids[at:]
    cap = len(free) + int(rng.integers(0, 4))
    head = int(rng.integers(0, 1 << 34)) if wrap else 0
    ring = np.full(cap, 10 ** 6)
    ring[(head + np.arange(len(free))) % cap] = free
    return new, held, table, ring, head, head + len(free)


def _run(case, tokens, in_place=True, **kw):
    pkv = _pkv()
    new, held, table, ring, head, tail = case
    dtable, state = _dev(table), _dev([head, tail, 0, 0], I64)
    err = torch.zeros(1, dtype=I32, device="cuda")
    out = None if in_place else torch.full((2,), 77, dtype=I64, device="cuda")
    got = pkv.build_step_metadata(_dev(new), _dev(held), dtable, _dev(ring), state, tokens,
                                  free_state_out=out, error_word=err, **kw)
    after = (state if in_place else out).tolist()
    if in_place:
        assert after[2:] == [0, 0]
    else:
        assert state.tolist() == [head, tail, 0, 0]
    return [dtable.tolist()] + [x.tolist() for x in got], after[:2], int(err)


@pytest.mark.parametrize("reqs, new_hi, held_hi, width, pad", [
    (1, 1, 0, 1, 0), (1, 1, 40, 4, 7), (1, 5000, 0, 400, 0), (3, 40, 40, 6, 5), (300, 1, 500, 32, 0),
    (511, 20, 100, 9, 3), (512, 1, 100, 9, 0), (513, 3, 90, 7, 1), (1500, 30, 60, 8, 100),
    (8192, 2, 30, 4, 9), (64, 600, 1000, 101, 1)])
@pytest.mark.parametrize("in_place", [True, False])
def test_parity(reqs, new_hi, held_hi, width, pad, in_place):
    rng = np.random.default_rng(reqs * 7 + new_hi)
    case = _case(rng, reqs, new_hi, held_hi, width)
    if reqs == 1:
        case[0][0] = max(1, case[0][0])
        case = _case(rng, reqs, new_hi, held_hi, width, spare=2 + new_hi // 16)
    new, held, table, ring, head, tail = case
    tokens = int(new.sum()) + pad
    want = mxfp4.step_metadata(new.tolist(), held.tolist(), table.tolist(), ring.tolist(), head, tail,
                               tokens)
    got, after, err = _run(case, tokens, in_place)
    assert err == 0
    assert got == list(want[:5])
    assert after == [want[5], tail]


@pytest.mark.parametrize("why", ["blocks", "row", "negative new", "negative held", "tokens", "state",
                                 "sum past 32 bits"])
def test_refused_steps_change_nothing(why):
    pkv = _pkv()
    rng = np.random.default_rng(3)
    new, held, table, ring, head, tail = _case(rng, 40, 30, 60, 7, spare=0)
    tokens, bit = int(new.sum()), pkv.ERR_METADATA
    if why == "blocks":
        tail, bit = tail - 1, pkv.ERR_NO_BLOCKS
    elif why == "row":
        table = table[:, :max(1, int((-(-(held + new) // 16)).max()) - 1)]
    elif why == "negative new":
        new[7] = -1
    elif why == "negative held":
        held[39] = -16
    elif why == "tokens":
        tokens -= 1
    elif why == "state":
        tail = head + len(ring) + 1
    elif why == "sum past 32 bits":
        new[:] = 2 ** 31 - 10 ** 6
    got, after, err = _run((new, held, table, ring, head, tail), tokens)
    assert err == bit
    assert after == [head, tail]
    assert got == [table.tolist(), [0] * 41, held.tolist(), [-1] * tokens, [0] * tokens]


def test_a_missing_held_block_is_flagged():
    pkv = _pkv()
    got, _, err = _run((np.array([3]), np.array([20]), np.array([[5, -1, -1]]), np.array([8]), 0, 1), 4)
    assert err == pkv.ERR_BLOCK_ID
    assert got[3] == [-1, -1, -1, -1] and got[4] == [20, 21, 22, 0]


def test_no_requests():
    pkv = _pkv()
    state = _dev([0, 0, 0, 0], I64)
    got = pkv.build_step_metadata(_dev([]), _dev([]), torch.empty(0, 4, dtype=I32, device="cuda"),
                                  _dev([]), state, 5)
    assert [x.tolist() for x in got] == [[0], [], [-1] * 5, [0] * 5]


def test_strided_table_and_width():
    """Rows of 4 entries inside rows of 9: the limit is the row's own width."""
    pkv = _pkv()
    wide = torch.full((2, 9), -7, dtype=I32, device="cuda")
    state = _dev([0, 8, 0, 0], I64)
    build = pkv.build_step_metadata
    err = torch.zeros(1, dtype=I32, device="cuda")
    build(_dev([64, 3]), _dev([0, 0]), wide[:, 2:6], _dev(range(8)), state, 80, error_word=err)
    assert wide.tolist() == [[-7, -7, 0, 1, 2, 3, -7, -7, -7], [-7, -7, 4] + [-7] * 6]
    build(_dev([1, 0]), _dev([64, 3]), wide[:, 2:6], _dev(range(8)), state, 80, error_word=err)
    assert int(err) == pkv.ERR_METADATA and state.tolist() == [5, 8, 0, 0]


def test_steps_follow_the_host_scheduler():
    """Prompts in chunks, then decodes: the device tables of every step are the
    scheduler's.  The whole sequence again as replays of one graph."""
    pkv = _pkv()
    lens = [37, 100, 5, 64]
    sched = pkv.Scheduler(8, 64, 32, 512, 16, 40, 12)
    for i, n in enumerate(lens):
        assert sched.add_request(i, n, 9)
    width = 12
    table = torch.full((4, width), -1, dtype=I32, device="cuda")
    ring, state = _dev(range(40)), _dev([0, 40, 0, 0], I64)
    held, new = _dev([0] * 4), _dev([0] * 4)
    buf = dict(query_start_loc=_dev([0] * 5), seq_lens=_dev([0] * 4), slot_mapping=_dev([0] * 64, I64),
               positions=_dev([0] * 64, I64), error_word=_dev([0]))
    gtable, gstate = table.clone(), state.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.build_step_metadata(new, held, gtable, ring, gstate, 64, **buf)
    for _ in range(14):
        plan = sched.step()
        if not plan["entries"]:
            break
        s, h = [0] * 4, [0] * 4
        for r in range(4):
            st = sched.request(r)
            h[r] = st["num_computed"]
        order = [r for r, _, _ in plan["entries"]]
        assert order == sorted(order)
        for r, n, before in plan["entries"]:
            s[r], h[r] = n, before
        bt, qsl, seq, nc, slots = sched.metadata(width)
        new.copy_(_dev(s))
        held.copy_(_dev(h))
        got = pkv.build_step_metadata(new, held, table, ring, state, 64)
        n = plan["num_tokens"]
        assert got[2][:n].tolist() == slots.tolist() and (got[2][n:] == -1).all()
        assert got[1][order].tolist() == seq.tolist()
        for row, r in enumerate(order):
            k = -(-int(seq[row]) // 16)
            assert table[r, :k].tolist() == bt[row, :k].tolist()
        graph.replay()
        assert int(buf["error_word"]) == 0
        for a, b in zip(got, (buf["query_start_loc"], buf["seq_lens"], buf["slot_mapping"],
                              buf["positions"])):
            assert torch.equal(a, b)
        assert torch.equal(table, gtable) and torch.equal(state, gstate)
        if sched.finish_step(True):
            break   # freed blocks go back to the host's list only


@pytest.mark.parametrize("hkv, group, d", [(2, 4, 128), (3, 2, 64)])
def test_serving_steps_end_to_end(hkv, group, d):
    """Prompt chunks and decodes of three requests: tables on the device, RoPE of
    Q and K, the 4-bit cache write, attention; every step against the oracle
    on the values that the cache holds, twice (a graph of the decode step)."""
    pkv = _pkv()
    rng = torch.Generator().manual_seed(d)
    H, width, nb = hkv * group, 10, 40
    table = torch.full((3, width), -1, dtype=I32, device="cuda")
    ring = torch.randperm(nb, generator=rng).int().cuda()
    state = _dev([0, nb, 0, 0], I64)
    kc, vc = pkv.new_cache_mxfp4(nb, hkv, d)
    bf_k = torch.zeros(1, 16, hkv, d, dtype=torch.bfloat16, device="cuda")  # RoPE's own cache, unused
    ang = torch.arange(256)[:, None] / 10000 ** (torch.arange(0, d, 2) / d)
    table_cs = torch.cat([ang.cos(), ang.sin()], 1).float().cuda().contiguous()
    ws = pkv.new_workspace_mxfp4(H, hkv, d)
    err = _dev([0])
    held = [0, 0, 0]
    for new in ([40, 7, 0], [30, 1, 20], [1, 1, 33], [1, 1, 1], [1, 0, 1]):
        T = sum(new) + 2
        # every row of the padded batch has a query, a key and a value
        qkv = torch.randn(T, H + 2 * hkv, d, generator=rng).to(torch.bfloat16).cuda()
        q, k, v = qkv[:, :H], qkv[:, H:H + hkv], qkv[:, H + hkv:]
        qsl, seq, slots, pos = pkv.build_step_metadata(_dev(new), _dev(held), table, ring, state, T,
                                                       error_word=err)
        skip = torch.full_like(slots, -1)
        pkv.rope_reshape_and_cache(pos, q, k, v, bf_k, bf_k.clone(), skip, table_cs, key_out=k,
                                   error_word=err)
        pkv.reshape_and_cache_mxfp4(k, v, kc, vc, slots, error_word=err)
        out = torch.full((T, H, d), 5.0, dtype=torch.bfloat16, device="cuda")
        pkv.paged_attention_varlen_mxfp4(q, kc, vc, table, qsl, seq, _dev(held), d ** -0.5, out=out,
                                         workspace=ws, max_query_len=max(new))
        assert int(err) == 0 and pkv.read_error_word(ws) == 0
        pools = kc.cpu().numpy(), vc.cpu().numpy()
        for r in range(3):
            a, n = sum(new[:r]), new[r]
            if n == 0:
                continue
            p = np.arange(held[r] + n)
            s = table[r].cpu().numpy()[p // 16].astype(np.int64) * 16 + p % 16
            kk, vv = (torch.from_numpy(mxfp4.read_rows(x, s, hkv, d, i == 0)) for i, x in enumerate(pools))
            ref = oa.causal_attention_request(q[a:a + n].cpu(), kk, vv, held[r], d ** -0.5)
            got = out[a:a + n].double().cpu()
            mean = oa.causal_attention_request(q[a:a + n].cpu(), kk, vv.abs(), held[r], d ** -0.5)
            # half a bfloat16 step, and f16 weights (2^-11) with room for the scores
            assert ((got - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -10 * mean).all()
            # the last token's K row: what the write rounded, within half a grid step
            last = k[a + n - 1].float().cpu().double()
            e = last.abs().unflatten(-1, (-1, 32)).amax(-1, keepdim=True)
            assert ((kk[-1] - last).abs().unflatten(-1, (-1, 32)) <= e / 4).all()
        assert (out[sum(new):] == 5.0).all()
        held = [h + n for h, n in zip(held, new)]
