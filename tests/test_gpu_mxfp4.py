"""GPU parity of the 4-bit paged cache: quantising write and read-back byte for
byte, attention within the bound derived in tests/mxfp4_support.py."""

import numpy as np
import pytest
import torch

from oracle import mxfp4
from tests.mxfp4_support import Step, check

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _pkv():
    import paged_kv_cache_36_gb300 as pkv
    return pkv


def _rows(rng, tokens, hkv, d):
    """Rows whose groups cover the whole range: ordinary ones, ties of the grid,
    zeros, tiny and huge ones, subnormals, NaN and infinities."""
    x = rng.standard_normal((tokens, hkv, d)).astype(np.float32)
    x *= np.exp2(rng.integers(-30, 30, (tokens, hkv, 1))).astype(np.float32)
    g = x.reshape(tokens, hkv, d // 32, 32)
    grid = np.array([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7], np.float32)
    for i, (t, h, b) in enumerate(np.ndindex(tokens, hkv, d // 32)):
        kind = i % 11
        if kind == 1:    # exact grid points and midpoints at some scale
            s = np.float32(2.0) ** rng.integers(-20, 20)
            g[t, h, b] = rng.permutation(np.concatenate([grid, -grid])) * s
        elif kind == 3:
            g[t, h, b] = 0
        elif kind == 5:  # below the smallest scale
            g[t, h, b] = rng.integers(-3, 4, 32) * np.float32(2.0 ** -127)
        elif kind == 7:
            g[t, h, b] = rng.standard_normal(32) * np.float32(2.0 ** 125)
        elif kind == 9 and i % 3 == 0:
            g[t, h, b, rng.integers(32)] = rng.choice([np.nan, np.inf, -np.inf])
    return torch.from_numpy(x)


@pytest.mark.parametrize("tokens, hkv, d, dtype, fused, pad", [
    (1, 1, 64, BF16, False, 0), (1, 8, 128, BF16, True, 0), (7, 2, 128, F32, True, 2),
    (33, 3, 64, BF16, True, 3), (18, 5, 128, BF16, False, 1), (9, 5, 64, F32, False, 0),
    (40, 1, 128, F32, False, 0)])
def test_write_is_the_oracle_byte_for_byte(tokens, hkv, d, dtype, fused, pad):
    pkv = _pkv()
    rng = np.random.default_rng(tokens * 100 + hkv * 10 + d)
    k, v = _rows(rng, tokens, hkv, d).to(dtype), _rows(rng, tokens, hkv, d).to(dtype)
    nb = tokens // 16 + 3
    pools = [rng.integers(0, 256, (nb, hkv * mxfp4.chunk_bytes(d)), dtype=np.uint8) for _ in "kv"]
    slots = rng.permutation(nb * 16)[:tokens].astype(np.int64)
    if pad:
        slots[rng.permutation(tokens)[:pad]] = -1
    kc, vc = (torch.from_numpy(p.copy()).cuda() for p in pools)
    dk, dv = k.cuda(), v.cuda()
    if fused:
        wide = torch.zeros(tokens, 4 * hkv, d, dtype=dtype, device="cuda")
        wide[:, hkv:2 * hkv], wide[:, 3 * hkv:] = dk, dv
        dk, dv = wide[:, hkv:2 * hkv], wide[:, 3 * hkv:]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.reshape_and_cache_mxfp4(dk, dv, kc, vc, torch.from_numpy(slots).cuda(), error_word=err)
    for t, s in enumerate(slots):
        if s >= 0:
            mxfp4.write_row(pools[0], int(s), k[t].double().numpy(), True)
            mxfp4.write_row(pools[1], int(s), v[t].double().numpy(), False)
    assert int(err) == 0
    assert np.array_equal(kc.cpu().numpy(), pools[0])
    assert np.array_equal(vc.cpu().numpy(), pools[1])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gather_reads_every_code_and_scale(d, dtype):
    """All 256 bytes as codes and as scales; outputs exact, NaN groups NaN."""
    pkv = _pkv()
    hkv, nb = 3, 40
    rng = np.random.default_rng(d)
    pools = [rng.integers(0, 256, (nb, hkv * mxfp4.chunk_bytes(d)), dtype=np.uint8) for _ in "kv"]
    slots = np.concatenate([rng.permutation(nb * 16), [5, 5]]).astype(np.int64)
    slots[3] = -2
    out = torch.full((2, len(slots), hkv + 1, d), 7.0, dtype=dtype, device="cuda")
    ko, vo = out[0][:, :hkv], out[1][:, 1:]
    pkv.gather_cache_mxfp4(*(torch.from_numpy(p).cuda() for p in pools),
                           torch.from_numpy(slots).cuda(), ko, vo)
    live = slots >= 0
    for o, pool, is_key in ((ko, pools[0], True), (vo, pools[1], False)):
        want = torch.from_numpy(mxfp4.read_rows(pool, slots[live], hkv, d, is_key))
        want = torch.where(want.abs() > torch.finfo(dtype).max, torch.copysign(
            torch.full_like(want, torch.inf), want), want)   # 6 x 2^126 and up
        assert torch.equal(o.cpu()[live].double().nan_to_num(nan=123.0), want.nan_to_num(nan=123.0))
        assert (o[3] == 7.0).all()
    assert (out[0][:, hkv:] == 7.0).all() and (out[1][:, :1] == 7.0).all()


def test_slots_past_the_pool():
    pkv = _pkv()
    hkv, d = 2, 64
    kc, vc = pkv.new_cache_mxfp4(2, hkv, d)
    slots = torch.tensor([32, 31, 1 << 40, -1], device="cuda")
    x = torch.ones(4, hkv, d, dtype=BF16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.reshape_and_cache_mxfp4(x, x, kc, vc, slots, error_word=err)
    assert int(err) == pkv.ERR_SLOT
    err.zero_()
    ko, vo = torch.full_like(x, 9.0), torch.full_like(x, 9.0)
    pkv.gather_cache_mxfp4(kc, vc, slots, ko, vo, error_word=err)
    assert int(err) == pkv.ERR_SLOT
    for o in (ko, vo):
        assert [float(o[t, 0, 0]) for t in range(4)] == [0.0, 1.0, 0.0, 9.0]


# --------------------------------------------------------------------- attention
DECODES = [
    # (requests, heads, hkv, d): contexts from one token on, odd ones, ends inside a block
    ([(1, 0)], 1, 1, 64),
    ([(1, 0), (1, 15), (1, 16), (1, 17)], 8, 2, 128),
    ([(1, 999)], 8, 2, 64),
    ([(1, p) for p in (0, 3, 31, 32, 63, 64, 65, 127, 500)], 32, 8, 128),
    ([(1, 4095), (0, 50), (1, 1), (1, 0), (1, 777)], 12, 3, 128),
    ([(1, p) for p in (100, 2000, 5, 300)], 35, 5, 64),     # 7 heads a KV head
    ([(1, 1500), (1, 12)], 32, 2, 128),                     # 16 heads a KV head
    ([(1, 640), (1, 33)], 11, 1, 64),
    ([(1, p % 97) for p in range(300)], 4, 4, 64),
    ([(1, 20000)], 8, 1, 128),
]
CHUNKS = [
    ([(2, 0)], 1, 1, 64),
    ([(7, 0), (128, 0), (3, 40)], 8, 2, 128),
    ([(129, 131)], 32, 8, 128),
    ([(100, 600), (33, 0), (1, 200), (0, 9), (1, 15)], 12, 3, 64),
    ([(64, 17), (1, 100), (65, 0)], 35, 5, 128),
    ([(37, 300), (1, 700)], 32, 2, 128),
    ([(300, 0), (2, 511)], 5, 1, 64),
    ([(512, 300)], 6, 2, 128),
]


@pytest.mark.parametrize("reqs, heads, hkv, d", DECODES + CHUNKS)
def test_attention(reqs, heads, hkv, d):
    pkv = _pkv()
    s = Step(len(reqs) * 1000 + heads, reqs, heads, hkv, d, stride_pad=1, table_pad=3).upload()
    ws = pkv.new_workspace_mxfp4(heads, hkv, d)
    got = pkv.paged_attention_varlen_mxfp4(*s.args(), workspace=ws,
                                           max_query_len=max(s.q_len))
    assert pkv.read_error_word(ws) == 0
    ref, tol = s.reference()
    check(got, ref, tol)
    # the hint left out
    again = pkv.paged_attention_varlen_mxfp4(*s.args(), workspace=ws)
    assert pkv.read_error_word(ws) == 0
    check(again, ref, tol)


@pytest.mark.parametrize("lo, hi", [(-40, 12), (-126, -100), (-60, 40), (-12, 12), (20, 21)])
@pytest.mark.parametrize("reqs", [[(1, 700), (1, 40)], [(90, 260)]])
def test_values_over_many_binades(lo, hi, reqs):
    """V scales 2^lo .. 2^hi side by side: in a row, in a tile, along a request."""
    pkv = _pkv()
    s = Step(hi - lo, reqs, 8, 2, 128)
    s.pools.scales(s.rng, np.concatenate(s.slots), lo, hi, k=False)
    s.upload()
    got = pkv.paged_attention_varlen_mxfp4(*s.args(), max_query_len=max(s.q_len))
    check(got, *s.reference())


@pytest.mark.parametrize("reqs", [[(1, 700), (1, 40)], [(90, 260), (1, 33)]])
def test_small_values_next_to_a_huge_one_with_no_weight(reqs):
    """One key that no query likes has values 2^60 times the others'."""
    pkv = _pkv()
    s = Step(11, reqs, 8, 2, 64)
    for slots in s.slots:
        one = slots[len(slots) // 2:len(slots) // 2 + 1]
        s.pools.scales(s.rng, one, 60, 60, k=False)
        # K of that token: far against every query (all queries share a direction)
        for h in range(2):
            c = h * mxfp4.chunk_bytes(64)
            blk, t = divmod(int(one[0]), 16)
            for dim in range(64):
                byte, high = mxfp4.code_place(t, dim, 64, True)
                code = 0xf if dim < 8 else 0x0
                old = int(s.pools.k[blk, c + byte])
                s.pools.k[blk, c + byte] = (old & 0x0f) | code << 4 if high else (old & 0xf0) | code
            s.pools.k[blk, c + mxfp4.scale_place(t, 0, 64, True)] = 127 + 4
            s.pools.k[blk, c + mxfp4.scale_place(t, 1, 64, True)] = 127
    s.q[:, :, :8] = 4.0
    s.upload()
    got = pkv.paged_attention_varlen_mxfp4(*s.args(), max_query_len=max(s.q_len))
    ref, tol = s.reference()
    # the token's weight is e^-384 at most: it may add nothing.  Leave its V
    # out of the bound: the result is compared as if it were an ordinary value.
    small = Step(11, reqs, 8, 2, 64)
    small.q[:, :, :8] = 4.0
    small.pools.k[:] = s.pools.k
    _, tol = small.reference()
    check(got, ref, tol)


@pytest.mark.parametrize("reqs", [[(1, 90), (1, 40)], [(20, 70), (1, 33)]])
@pytest.mark.parametrize("lo, hi", [(-120, -110), (4, 8), (-20, 7)])
def test_keys_over_many_binades(lo, hi, reqs):
    pkv = _pkv()
    s = Step(5, reqs, 4, 2, 64)
    s.pools.scales(s.rng, np.concatenate(s.slots), lo, hi, v=False)
    s.upload()
    got = pkv.paged_attention_varlen_mxfp4(*s.args(), max_query_len=max(s.q_len))
    check(got, *s.reference())


@pytest.mark.parametrize("factor", [1e30, 1e-30, 1e-3])
@pytest.mark.parametrize("reqs", [[(1, 90)], [(20, 70)]])
def test_queries_far_from_one(factor, reqs):
    """Large queries with a scale that undoes it, and the reverse."""
    pkv = _pkv()
    s = Step(6, reqs, 4, 2, 64)
    s.q = (s.q.float() * factor).to(BF16)
    s.q[0, 0] = 0
    s.scale = 0.125 / factor
    s.upload()
    got = pkv.paged_attention_varlen_mxfp4(*s.args(), max_query_len=max(s.q_len))
    check(got, *s.reference())


@pytest.mark.parametrize("scale", [-0.2, 0.0, 1e-30, 2.0])
@pytest.mark.parametrize("reqs", [[(1, 90), (1, 40)], [(20, 70)]])
def test_scales_of_the_scores(scale, reqs):
    pkv = _pkv()
    s = Step(12, reqs, 4, 2, 64)
    s.scale = scale
    s.upload()
    got = pkv.paged_attention_varlen_mxfp4(*s.args(), max_query_len=max(s.q_len))
    check(got, *s.reference())


@pytest.mark.parametrize("is_key", [True, False])
@pytest.mark.parametrize("reqs", [[(1, 90), (1, 40)], [(20, 70), (1, 40)]])
def test_a_nan_group_stays_with_its_rows(reqs, is_key):
    """A NaN group of a visible token makes NaN what depends on it and nothing else."""
    pkv = _pkv()
    s = Step(7, reqs, 4, 2, 128)
    tok = 85 if reqs[0][0] > 1 else 30
    slot = int(s.slots[0][tok])
    pool = s.pools.k if is_key else s.pools.v
    pool[slot // 16, mxfp4.chunk_bytes(128) + mxfp4.scale_place(slot % 16, 2, 128, is_key)] = 255
    for dim in range(64, 96):   # what the cache write stores: zero codes
        byte, _ = mxfp4.code_place(slot % 16, dim, 128, is_key)
        pool[slot // 16, mxfp4.chunk_bytes(128) + byte] = 0
    s.nan = (0,)
    s.upload()
    got = pkv.paged_attention_varlen_mxfp4(*s.args(), max_query_len=max(s.q_len)).double().cpu()
    ref, tol = s.reference()
    bad = torch.zeros_like(ref, dtype=torch.bool)
    first = max(0, tok - s.past[0])
    bad[first:s.q_len[0], 2:, (slice(None) if is_key else slice(64, 96))] = True
    assert torch.isnan(ref[bad]).all() and torch.isfinite(ref[~bad]).all()
    assert torch.isnan(got[bad]).all()
    check(got, ref, tol, rows=~bad)


def test_bad_blocks_and_bad_metadata():
    pkv = _pkv()
    reqs = [(1, 90), (40, 70), (1, 33), (5, 5), (1, 20)]
    s = Step(8, reqs, 8, 2, 64)
    ref, tol = s.reference()
    for r, col, bad in ((0, 2, -1), (1, 3, 10 ** 6)):
        t = Step(8, reqs, 8, 2, 64)
        t.table[r, col] = bad
        t.upload()
        ws = pkv.new_workspace_mxfp4(8, 2, 64)
        got = pkv.paged_attention_varlen_mxfp4(*t.args(), workspace=ws)
        assert pkv.read_error_word(ws) == pkv.ERR_BLOCK_ID
        keep = torch.ones(t.T, dtype=torch.bool)
        keep[int(t.qsl[r]):int(t.qsl[r + 1])] = False
        check(got, ref, tol, rows=keep)
        # the bad block reads as zeros
        zero = Step(8, reqs, 8, 2, 64)
        blk = int(zero.table[r, col])
        zero.pools.k[blk] = 0
        zero.pools.v[blk] = 0
        check(got, *zero.reference(), rows=~keep)
    for r, field, bad in ((0, "dseq", 90), (1, "dseq", 111), (2, "dpast", -1), (3, "dseq", 10 ** 9),
                          (1, "dpast", -40)):
        t = Step(8, reqs, 8, 2, 64).upload()
        getattr(t, field)[r] = bad
        if field == "dpast":
            t.dseq[r] = bad + t.q_len[r]
        ws = pkv.new_workspace_mxfp4(8, 2, 64)
        out = torch.full_like(t.dq, 3.0)
        got = pkv.paged_attention_varlen_mxfp4(*t.args(), out=out, workspace=ws)
        assert pkv.read_error_word(ws) == pkv.ERR_METADATA
        keep = torch.ones(t.T, dtype=torch.bool)
        keep[int(t.qsl[r]):int(t.qsl[r + 1])] = False
        check(got, ref, tol, rows=keep)
        assert (got.cpu()[~keep] == 3.0).all()


def test_rows_behind_the_last_request_are_left_alone():
    pkv = _pkv()
    s = Step(9, [(1, 30), (3, 5)], 8, 2, 64).upload()
    q = torch.cat([s.dq, torch.full((5, 8, 64), float("nan"), dtype=BF16, device="cuda")])
    out = torch.full_like(q, 4.0)
    args = (q,) + s.args()[1:]
    got = pkv.paged_attention_varlen_mxfp4(*args, out=out)
    ref, tol = s.reference()
    check(got[:4], ref, tol)
    assert (got[4:] == 4.0).all()
    # no requests, or none with rows
    none = torch.zeros(3, dtype=torch.int32, device="cuda")
    pkv.paged_attention_varlen_mxfp4(q, s.kc, s.vc, s.bt, none, s.dpast, s.dpast, 1.0, out=out)
    assert (out[4:] == 4.0).all()


def test_decode_hint_leaves_longer_rows():
    pkv = _pkv()
    s = Step(10, [(1, 30), (3, 5), (1, 100)], 8, 2, 64).upload()
    out = torch.full_like(s.dq, 4.0)
    got = pkv.paged_attention_varlen_mxfp4(*s.args(), out=out, max_query_len=1)
    ref, tol = s.reference()
    check(got, ref, tol, rows=torch.tensor([0, 4]))
    assert (got[1:4] == 4.0).all()


def test_one_workspace_through_many_batches_and_repeats():
    """The same workspace through batches of other sizes, twice each, equal bits."""
    pkv = _pkv()
    ws = pkv.new_workspace_mxfp4(32, 8, 128)
    steps = [Step(20 + i, reqs, 32, 8, 128).upload() for i, reqs in enumerate(
        [[(1, 3000)], [(1, 50)] * 40, [(60, 10), (1, 2000)], [(1, 0)], [(1, 700), (1, 3)]])]
    first = [pkv.paged_attention_varlen_mxfp4(*s.args(), workspace=ws).clone() for s in steps]
    for s, f in zip(steps, first):
        check(f, *s.reference())
    for s, f in list(zip(steps, first))[::-1]:
        assert torch.equal(pkv.paged_attention_varlen_mxfp4(*s.args(), workspace=ws), f)
    assert pkv.read_error_word(ws) == 0


def test_graph_replay_and_another_stream():
    pkv = _pkv()
    s = Step(31, [(1, 900), (17, 40), (1, 12)], 8, 2, 64).upload()
    ref, tol = s.reference()
    ws = pkv.new_workspace_mxfp4(8, 2, 64)
    out = torch.zeros_like(s.dq)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pkv.paged_attention_varlen_mxfp4(*s.args(), workspace=ws, out=out, stream=side)
    side.synchronize()
    check(out, ref, tol)
    # workspace and out made by the call, on the call's stream
    got = pkv.paged_attention_varlen_mxfp4(*s.args(), stream=side)
    side.synchronize()
    check(got, ref, tol)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pkv.paged_attention_varlen_mxfp4(*s.args(), workspace=ws, out=out)
        graphs.append(g)
    want = got.clone()
    for g in graphs * 2:
        out.zero_()
        g.replay()
        assert torch.equal(out, want)


def test_offsets_past_32_bits():
    """Blocks beyond 2^31 bytes of a pool."""
    pkv = _pkv()
    hkv, d = 8, 128
    nb = 260000
    assert nb * pkv.mxfp4_block_bytes(hkv, d) > 1 << 31
    s = Step(41, [(1, 200), (30, 70)], 8, 8, 128)
    small = s.pools
    s.upload()
    shift = nb - small.k.shape[0]
    kc, vc = pkv.new_cache_mxfp4(nb, hkv, d)
    kc[shift:], vc[shift:] = s.kc, s.vc
    got = pkv.paged_attention_varlen_mxfp4(s.dq, kc, vc, s.bt + shift, *s.args()[4:])
    check(got, *s.reference())
    slots = torch.tensor([(nb - 1) * 16 + 3], device="cuda")
    x = torch.randn(1, hkv, d, device="cuda")
    pkv.reshape_and_cache_mxfp4(x, x, kc, vc, slots)
    ko, vo = torch.empty_like(x), torch.empty_like(x)
    pkv.gather_cache_mxfp4(kc, vc, slots, ko, vo)
    assert torch.equal(ko, vo)
    # with amax in [4 s, 8 s) of a group's scale s: half a step is s at most, and
    # saturation at 6 s takes off amax - 6 s; both are amax / 4 at most
    assert ((ko - x).abs().unflatten(-1, (-1, 32))
            <= x.abs().unflatten(-1, (-1, 32)).amax(-1, keepdim=True) / 4).all()
    pool = kc[-1:].cpu().numpy()
    assert torch.equal(ko.cpu().double(), torch.from_numpy(mxfp4.read_rows(pool, [3], hkv, d, True)))


def test_copy_blocks_moves_4_bit_blocks():
    pkv = _pkv()
    s = Step(51, [(1, 200)], 8, 2, 64).upload()
    nb = s.kc.shape[0]
    kc, vc = pkv.new_cache_mxfp4(nb + 7, 2, 64)
    to = torch.randperm(nb + 7)[:s.width].int()
    pairs = torch.stack([s.bt[0].cpu(), to], 1).contiguous().cuda()
    pkv.copy_blocks(s.kc, s.vc, kc, vc, pairs)
    got = pkv.paged_attention_varlen_mxfp4(s.dq, kc, vc, to.cuda()[None], *s.args()[4:])
    check(got, *s.reference())
