"""GPU parity of the 8-bit paged cache: the quantising write (alone and with RoPE) and the
read-back."""

import numpy as np
import pytest
import torch

from oracle import fp8

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _pkv():
    import paged_kv_cache_36_gb300 as pkv
    return pkv


def _rows(rng, tokens, hkv, d):
    """Rows over the whole range: ordinary ones, ties of the grid, zeros, tiny and huge ones,
    subnormals, NaN and infinities."""
    x = rng.standard_normal((tokens, hkv, d)).astype(np.float32)
    x *= np.exp2(rng.integers(-12, 12, (tokens, hkv, 1))).astype(np.float32)
    grid = np.array([float(g) for g in fp8.GRID])
    ties = np.concatenate([grid, (grid[1:] + grid[:-1]) / 2, [456.0, 464.0, 480.0]]).astype(np.float32)
    for i, (t, h) in enumerate(np.ndindex(tokens, hkv)):
        kind = i % 13
        if kind == 1:
            s = np.float32(2.0) ** rng.integers(-20, 20)
            x[t, h] = rng.choice(ties, d) * rng.choice(np.array([1, -1], np.float32), d) * s
        elif kind == 3:
            x[t, h] = 0
        elif kind == 5:  # below the smallest scale
            x[t, h] = rng.integers(-3, 4, d) * np.float32(2.0 ** -127)
        elif kind == 7 and i % 2:
            x[t, h] = rng.standard_normal(d) * np.float32(2.0 ** 125)
        elif kind == 9:
            x[t, h, rng.integers(d)] = rng.choice([np.nan, np.inf, -np.inf])
    return torch.from_numpy(x)


def _fused(x, before, after):
    wide = torch.zeros(x.shape[0], before + x.shape[1] + after, x.shape[2], dtype=x.dtype, device="cuda")
    wide[:, before:before + x.shape[1]] = x.cuda()
    return wide[:, before:before + x.shape[1]]


def _pools(rng, nb, hkv, d):
    return [rng.integers(0, 256, (nb, hkv * fp8.chunk_bytes(d)), dtype=np.uint8) for _ in "kv"]


def _same(cache, pool, hkv, d):
    """Byte for byte; of the codes for NaN either sign."""
    got = cache.cpu().numpy()
    view = lambda a: a.reshape(len(a), hkv, -1)[..., :16 * d] & 127  # noqa: E731
    nan = np.zeros_like(got, dtype=bool)
    nan.reshape(len(got), hkv, -1)[..., :16 * d] = (view(got) == 127) & (view(pool) == 127)
    assert np.array_equal(got[~nan], pool[~nan])


@pytest.mark.parametrize("tokens, hkv, d, dtype, fused, pad, order", [
    (1, 1, 64, BF16, False, 0, "blocks"), (1, 8, 128, BF16, True, 0, "blocks"),
    (7, 2, 128, F32, True, 2, "random"), (33, 3, 64, BF16, True, 3, "random"),
    (16, 5, 128, BF16, False, 0, "blocks"), (50, 1, 128, F32, False, 1, "blocks"),
    (40, 5, 64, F32, False, 0, "reversed"), (300, 1, 64, BF16, False, 5, "blocks"),
    (700, 1, 64, BF16, True, 0, "random"), (1300, 1, 64, BF16, False, 3, "woven"), (1900, 1, 64, F32, False, 0, "random")])
def test_write_is_the_oracle_byte_for_byte(tokens, hkv, d, dtype, fused, pad, order):
    """Two calls into noise, the second behind the rows of the first: restarted blocks,
    blocks whose scale grows, blocks whose scale stays."""
    pkv = _pkv()
    rng = np.random.default_rng(tokens * 100 + hkv * 10 + d)
    nb = 2 * tokens // 16 + 3
    pools = _pools(rng, nb, hkv, d)
    kc, vc = (torch.from_numpy(p.copy()).cuda() for p in pools)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    start = int(rng.integers(0, 16))
    every = (rng.permutation(nb)[:, None] * 16 + np.arange(16)).reshape(-1)
    if order == "random":
        every = rng.permutation(nb * 16)
    for call in range(2):
        slots = every[start + call * tokens:start + (call + 1) * tokens].astype(np.int64)
        if order == "reversed":
            slots = slots[::-1].copy()
        if order == "woven":    # neighbours from two blocks in turn
            slots = slots[np.argsort(np.arange(tokens) % 16 + np.arange(tokens) // 32 * 32, kind="stable")]
        if pad:
            slots[rng.permutation(tokens)[:pad]] = -1
        k, v = _rows(rng, tokens, hkv, d).to(dtype), _rows(rng, tokens, hkv, d).to(dtype)
        dk, dv = (_fused(x, hkv, 2 * hkv) if fused else x.cuda() for x in (k, v))
        pkv.reshape_and_cache_fp8(dk, dv, kc, vc, torch.from_numpy(slots).cuda(), error_word=err)
        fp8.write(pools[0], slots, k.double().numpy(), True)
        fp8.write(pools[1], slots, v.double().numpy(), False)
    assert int(err) == 0
    _same(kc, pools[0], hkv, d)
    _same(vc, pools[1], hkv, d)


def test_token_by_token_as_a_decode_does():
    """40 calls of one token each, louder and louder, into two blocks and a half."""
    pkv = _pkv()
    rng = np.random.default_rng(5)
    hkv, d = 2, 128
    pools = _pools(rng, 4, hkv, d)
    kc, vc = (torch.from_numpy(p.copy()).cuda() for p in pools)
    table = [2, 0, 3]
    for t in range(40):
        slot = np.array([table[t // 16] * 16 + t % 16])
        k, v = (torch.from_numpy(rng.standard_normal((1, hkv, d)).astype(np.float32) * 1.3 ** t) for _ in "kv")
        pkv.reshape_and_cache_fp8(k.cuda(), v.cuda(), kc, vc, torch.from_numpy(slot).cuda())
        fp8.write(pools[0], slot, k.double().numpy(), True)
        fp8.write(pools[1], slot, v.double().numpy(), False)
    _same(kc, pools[0], hkv, d)
    _same(vc, pools[1], hkv, d)


@pytest.mark.parametrize("count", [40, 1000])
def test_the_last_of_equal_slots_counts(count):
    """`count` tokens for 9 slots of two blocks, with padding and slots past the pool."""
    pkv = _pkv()
    rng = np.random.default_rng(count)
    hkv, d = 1, 64
    pools = _pools(rng, 3, hkv, d)
    kc, vc = (torch.from_numpy(p.copy()).cuda() for p in pools)
    slots = rng.choice([3, 4, 9, 15, 16, 20, 21, 30, 31, -1, 48, 1 << 40], count).astype(np.int64)
    k, v = _rows(rng, count, hkv, d), _rows(rng, count, hkv, d)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.reshape_and_cache_fp8(k.cuda(), v.cuda(), kc, vc, torch.from_numpy(slots).cuda(), error_word=err)
    slots[slots >= 48] = -1
    fp8.write(pools[0], slots, k.double().numpy(), True)
    fp8.write(pools[1], slots, v.double().numpy(), False)
    assert int(err) == pkv.ERR_SLOT
    _same(kc, pools[0], hkv, d)
    _same(vc, pools[1], hkv, d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gather_reads_every_code_and_scale(d, dtype):
    pkv = _pkv()
    hkv, nb = 3, 40
    rng = np.random.default_rng(d)
    pools = _pools(rng, nb, hkv, d)
    for p in pools:
        p.reshape(nb, hkv, -1)[..., 16 * d] = rng.permutation(np.arange(nb * hkv) * 2 % 256).reshape(nb, hkv)
    slots = rng.permutation(nb * 16).astype(np.int64)[:501]
    slots[[3, 77]] = -1, nb * 16
    wide = [torch.full((501, 2 * hkv, d), 7.0, dtype=dtype, device="cuda") for _ in "kv"]
    outs = [w[:, hkv:] for w in wide]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kc, vc = (torch.from_numpy(p).cuda() for p in pools)
    pkv.gather_cache_fp8(kc, vc, torch.from_numpy(slots).cuda(), *outs, error_word=err)
    assert int(err) == pkv.ERR_SLOT
    for out, pool, key, w in zip(outs, pools, (True, False), wide):
        want = fp8.read_rows(pool, np.clip(slots, 0, nb * 16 - 1), hkv, d, key)
        want[3], want[77] = 7.0, 0.0
        assert np.array_equal(out.double().cpu().numpy(), want, equal_nan=True)
        assert (w[:, :hkv] == 7).all()


def _rotated(x, pos, table, rd, neox):
    """float64 rotation of [T, heads, D]."""
    y = x.double().clone()
    cos, sin = (table[pos, i * rd // 2:(i + 1) * rd // 2].double()[:, None] for i in (0, 1))
    a, b = (slice(0, rd // 2), slice(rd // 2, rd)) if neox else (slice(0, rd, 2), slice(1, rd, 2))
    xa, xb = x[..., a].double(), x[..., b].double()
    y[..., a], y[..., b] = xa * cos - xb * sin, xb * cos + xa * sin
    return y


@pytest.mark.parametrize("tokens, heads, hkv, d, rd, neox, dtype, in_place", [
    (1, 4, 1, 64, 64, True, BF16, True), (9, 8, 2, 128, 128, True, BF16, False),
    (33, 6, 3, 128, 64, False, BF16, False), (17, 5, 5, 64, 16, True, BF16, True),
    (40, 4, 2, 128, 96, True, F32, False), (20, 3, 1, 64, 24, True, F32, True),
    (50, 4, 4, 64, 8, False, BF16, False), (700, 2, 1, 128, 32, False, F32, True),
    (600, 7, 1, 64, 32, True, BF16, True)])
def test_rope_and_write(tokens, heads, hkv, d, rd, neox, dtype, in_place):
    """Rotated queries within the rounding of two products, a sum and the type: 3 2^-24
    (|x_a| + |x_b|) and half a step; codes those of the rotated key within its rounding
    (3 2^-24 of the pair, so at most one code away and then from a border that near)."""
    pkv = _pkv()
    rng = np.random.default_rng(tokens + rd)
    rows = torch.from_numpy(rng.standard_normal((tokens, heads + 2 * hkv, d)).astype(np.float32)).to(dtype).cuda()
    q, k, v = rows[:, :heads], rows[:, heads:heads + hkv], rows[:, heads + hkv:]
    before = rows.clone().cpu()
    table = torch.from_numpy(fp8.cos_sin(1000, rd).astype(np.float32))
    pos = rng.integers(0, 1000, tokens).astype(np.int64)
    nb = tokens // 16 + 3
    slots = (rng.permutation(nb)[:, None] * 16 + np.arange(16)).reshape(-1)[5:5 + tokens].astype(np.int64)
    if tokens > 5:
        pos[2], pos[4] = -1, 1000           # neither rotated nor written
        slots[3] = -1                       # rotated, not written
    kc, vc = pkv.new_cache_fp8(nb, hkv, d)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = None if in_place else torch.full((tokens, heads, d), 9.0, dtype=dtype, device="cuda")
    pkv.rope_reshape_and_cache_fp8(torch.from_numpy(pos).cuda(), q, k, v, kc, vc, torch.from_numpy(slots).cuda(),
                                   table.cuda(), is_neox=neox, query_out=out, error_word=err)
    assert int(err) == (pkv.ERR_POSITION if tokens > 5 else 0)
    bad = (pos < 0) | (pos >= 1000)
    safe = np.where(bad, 0, pos)
    half = torch.finfo(dtype).eps / 2

    def near(x):    # what a rotated value may be off by, before it is rounded to its type
        a = x.double().abs()
        m = torch.zeros_like(a)
        i, j = (slice(0, rd // 2), slice(rd // 2, rd)) if neox else (slice(0, rd, 2), slice(1, rd, 2))
        m[..., i] = m[..., j] = 3 * 2.0 ** -24 * (a[..., i] + a[..., j])
        return m

    want = _rotated(before[:, :heads], safe, table, rd, neox)
    got = (q if in_place else out).double().cpu()
    tol = near(before[:, :heads]) + half * want.abs() * (1 + 2.0 ** -20)
    ok = torch.from_numpy(~bad)
    assert ((got - want).abs() <= tol)[ok].all()
    assert torch.equal(got[~ok], before[:, :heads].double()[~ok] if in_place else torch.full_like(got[~ok], 9.0))
    kept = rows.cpu()[:, heads:]
    assert torch.equal(kept, before[:, heads:])          # keys and values are only read

    live = np.where(bad, -1, slots)
    kk = _rotated(before[:, heads:heads + hkv], safe, table, rd, neox)
    shape = (nb, hkv * fp8.chunk_bytes(d))
    pool = np.zeros(shape, np.uint8)
    fp8.write(pool, live, before[:, heads + hkv:].double().numpy(), False)
    _same(vc, pool, hkv, d)
    at = np.flatnonzero(live >= 0)
    back = fp8.read_rows(kc.cpu().numpy(), live[at], hkv, d, True)
    scale = kc.cpu().numpy().reshape(nb, hkv, -1)[live[at] // 16][..., 16 * d].astype(int)
    for i, t in enumerate(at):
        for h in range(hkv):
            x, step = kk[t, h].numpy(), 2.0 ** (scale[i, h] - 127)
            # half a step of the code's binade, and the rotation's own rounding
            room = np.maximum(np.abs(x) * 2.0 ** -4, step * 2.0 ** -10) * (1 + 2.0 ** -20) + near(before[t:t + 1, heads + h])[0].numpy()
            assert (np.abs(back[i, h] - x) <= room).all()
    for blk in np.unique(live[at] // 16):
        for h in range(hkv):
            xs = np.abs(kk[torch.from_numpy(np.flatnonzero(live // 16 == blk))][:, h].numpy())
            e = int(kc.cpu().numpy().reshape(nb, hkv, -1)[blk, h, 16 * d])
            assert fp8.scale_of([xs.max() * (1 - 2.0 ** -20)]) <= e <= fp8.scale_of([xs.max() * (1 + 2.0 ** -20)])


def test_other_stream_and_copied_blocks():
    """Write on a stream of its own, copy the blocks, read the copies."""
    pkv = _pkv()
    rng = np.random.default_rng(1)
    hkv, d, T = 2, 64, 64
    kc, vc = pkv.new_cache_fp8(8, hkv, d)
    k, v = (torch.from_numpy(rng.standard_normal((T, hkv, d)).astype(np.float32)).cuda() for _ in "kv")
    slots = torch.arange(T, device="cuda")
    pairs = torch.tensor([[i, 7 - i] for i in range(4)], dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    pkv.reshape_and_cache_fp8(k, v, kc, vc, slots, stream=s)
    pkv.copy_blocks(kc, vc, kc, vc, pairs, stream=s)
    outs = [[torch.empty(T, hkv, d, device="cuda") for _ in "kv"] for _ in range(2)]
    there = (7 - slots // 16) * 16 + slots % 16
    torch.cuda.current_stream().synchronize()
    pkv.gather_cache_fp8(kc, vc, slots, *outs[0], stream=s)
    pkv.gather_cache_fp8(kc, vc, there, *outs[1], stream=s)
    s.synchronize()
    for a, b, x in zip(*outs, (k, v)):
        assert torch.equal(a, b) and ((a - x).abs() <= x.abs() * 2.0 ** -4 + 2.0 ** -12).all()


def test_blocks_of_more_than_two_to_the_31_bytes():
    """As many KV heads as are allowed: offsets inside a block pass 2^31."""
    pkv = _pkv()
    hkv, d = 1 << 20, 128
    kc, vc = pkv.new_cache_fp8(1, hkv, d)
    assert kc.shape[1] > 1 << 31
    gen = torch.Generator(device="cuda").manual_seed(0)
    k, v = (torch.randn(2, hkv, d, generator=gen, device="cuda").to(BF16) for _ in "kv")
    for slots in ([0, 5], [9, 2]):      # (the second call's rows join the first's)
        slots = torch.tensor(slots, device="cuda")
        pkv.reshape_and_cache_fp8(k, v, kc, vc, slots)
        outs = [torch.empty_like(k) for _ in "kv"]
        pkv.gather_cache_fp8(kc, vc, slots, *outs)
        for out, x in zip(outs, (k, v)):
            for h in range(0, hkv, 1 << 17):
                a, b = out[:, h:h + (1 << 17)].float(), x[:, h:h + (1 << 17)].float()
                # half a code's step, 2^-10 of a scale of at most 2^-5 below the codes' normal range
                assert ((a - b).abs() <= b.abs() * 2.0 ** -4 + 2.0 ** -15).all()
