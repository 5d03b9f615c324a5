"""The 8-bit cache's write and read-back of some thousand tokens: windows of several tokens, the
search of two slots at a load, and blocks that are read whole."""

import numpy as np
import pytest
import torch

from oracle import fp8
from tests.fp8_support import write_many
from tests.test_gpu_fp8_cache import BF16, F32, _fused, _pkv, _pools, _rotated, _same

pytestmark = pytest.mark.gpu


def _slots(rng, order, tokens, nb, at):
    """A call's slots: those of `tokens` from the at-th on, of blocks that follow one another in
    no order."""
    every = (rng.permutation(nb)[:, None] * 16 + np.arange(16)).reshape(-1)
    if order == "shuffled":
        return rng.permutation(every)[:tokens]
    slots = every[at:at + tokens]
    if order == "requests":         # twenty, that begin inside blocks
        slots = np.concatenate([x[:len(x) - i % 3] for i, x in enumerate(np.array_split(every[at:at + tokens + 40], 20))])[:tokens]
    elif order == "duplicates":     # some slots again, near and far from where they were
        slots[rng.permutation(tokens)[:tokens // 8]] = rng.choice(slots, tokens // 8)
        slots[1::97] = slots[::97][:len(slots[1::97])]
    elif order == "reversed":
        slots = slots[::-1]
    return slots.copy()


def _values(rng, tokens, hkv, d):
    x = rng.standard_normal((tokens, hkv, d)).astype(np.float32)
    x *= np.exp2(rng.integers(-9, 9, (tokens, hkv, 1))).astype(np.float32)
    x[rng.integers(0, tokens, 9), 0, rng.integers(0, d, 9)] = rng.choice([np.nan, np.inf, -np.inf], 9)
    return torch.from_numpy(x)


@pytest.mark.parametrize("tokens, hkv, d, dtype, order, aligned", [
    (2500, 1, 64, BF16, "requests", True), (3700, 2, 128, BF16, "blocks", True), (4095, 1, 64, F32, "requests", True),
    (4096, 1, 64, BF16, "blocks", True), (4097, 2, 64, BF16, "duplicates", False), (5000, 3, 64, F32, "requests", True),
    (5000, 1, 128, BF16, "shuffled", True), (8200, 1, 64, BF16, "duplicates", True), (6001, 1, 64, BF16, "reversed", False),
    (9000, 8, 128, BF16, "requests", True)])
def test_write(tokens, hkv, d, dtype, order, aligned):
    """Two calls into noise, the second behind the rows of the first, byte for byte."""
    pkv = _pkv()
    rng = np.random.default_rng(tokens + d)
    nb = 2 * tokens // 16 + 8
    pools = _pools(rng, nb, hkv, d)
    kc, vc = (torch.from_numpy(p.copy()).cuda() for p in pools)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    seed, start = int(rng.integers(1 << 30)), int(rng.integers(1, 16))
    for call in range(2):
        slots = _slots(np.random.default_rng(seed), order, tokens, nb, start + call * (tokens - 40))
        slots[rng.permutation(tokens)[:7]] = -1
        past = rng.permutation(tokens)[:3]
        slots[past] = nb * 16 + np.array([0, 5, 1 << 40])
        k, v = (_values(rng, tokens, hkv, d).to(dtype) for _ in "kv")
        room = torch.full((tokens + 1,), -1, dtype=torch.int64, device="cuda")
        ds = room[:tokens] if aligned else room[1:]
        ds.copy_(torch.from_numpy(slots))
        assert (ds.data_ptr() % 16 == 0) == aligned
        pkv.reshape_and_cache_fp8(_fused(k, 1, 2), _fused(v, 0, 1), kc, vc, ds, error_word=err)
        slots[past] = -1
        write_many(pools[0], slots, k.double().numpy(), True)
        write_many(pools[1], slots, v.double().numpy(), False)
    assert int(err) == pkv.ERR_SLOT
    _same(kc, pools[0], hkv, d)
    _same(vc, pools[1], hkv, d)


@pytest.mark.parametrize("tokens, heads, hkv, d, rd, neox, dtype, order", [
    (2500, 4, 2, 128, 128, True, BF16, "requests"), (4100, 2, 1, 64, 32, False, F32, "shuffled"),
    (5000, 3, 1, 64, 64, True, F32, "requests"), (2048, 6, 2, 64, 16, False, BF16, "blocks")])
def test_rope_and_write(tokens, heads, hkv, d, rd, neox, dtype, order):
    """Rotated queries and keys within the rounding of two products and a sum, 3 2^-24 of the pair,
    and half a step of the type or the code; values byte for byte."""
    pkv = _pkv()
    rng = np.random.default_rng(tokens)
    rows = torch.from_numpy(rng.standard_normal((tokens, heads + 2 * hkv, d)).astype(np.float32)).to(dtype).cuda()
    before = rows.clone().cpu()
    table = torch.from_numpy(fp8.cos_sin(9000, rd).astype(np.float32))
    pos = rng.integers(0, 9000, tokens)
    nb = tokens // 16 + 8
    slots = _slots(rng, order, tokens, nb, 5)
    slots[3::500], pos[4::700] = -1, 9000
    kc, vc = pkv.new_cache_fp8(nb, hkv, d)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    up = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    q, k, v = rows[:, :heads], rows[:, heads:heads + hkv], rows[:, heads + hkv:]
    pkv.rope_reshape_and_cache_fp8(up(pos), q, k, v, kc, vc, up(slots), table.cuda(), is_neox=neox, error_word=err)
    assert int(err) == pkv.ERR_POSITION
    ok = pos < 9000
    want = _rotated(before[:, :heads + hkv], np.where(ok, pos, 0), table, rd, neox)
    a = before[:, :heads + hkv].double().abs()
    near = torch.zeros_like(a)
    i, j = (slice(0, rd // 2), slice(rd // 2, rd)) if neox else (slice(0, rd, 2), slice(1, rd, 2))
    near[..., i] = near[..., j] = 3 * 2.0 ** -24 * (a[..., i] + a[..., j])
    half = torch.finfo(dtype).eps / 2 * want.abs() * (1 + 2.0 ** -20)
    got = rows.cpu().double()[:, :heads]
    assert ((got - want[:, :heads]).abs() <= (near + half)[:, :heads])[ok].all()
    assert torch.equal(got[~ok], before[:, :heads].double()[~ok])

    live = np.where(ok, slots, -1)
    pools = [np.zeros((nb, hkv * fp8.chunk_bytes(d)), np.uint8) for _ in "kv"]
    write_many(pools[0], live, want[:, heads:].numpy(), True)
    write_many(pools[1], live, before[:, heads + hkv:].double().numpy(), False)
    _same(vc, pools[1], hkv, d)
    # the keys' scales, but where a block's largest is as near to a border as the rotation's rounding
    scale, mine = (p.reshape(nb, hkv, -1)[..., 16 * d].astype(int) for p in (kc.cpu().numpy(), pools[0]))
    assert (np.abs(scale - mine) <= 1).all() and (scale != mine).mean() < 0.01
    at = np.flatnonzero(live >= 0)
    back = fp8.read_rows(kc.cpu().numpy(), live[at], hkv, d, True)
    x = want[at, heads:].numpy()
    step = np.exp2(scale[live[at] // 16] - 127.0)[..., None]
    room = np.maximum(np.abs(x) * 2.0 ** -4, step * 2.0 ** -10) * (1 + 2.0 ** -20) + near[at, heads:].numpy()
    assert (np.abs(back - x) <= room).all()


@pytest.mark.parametrize("tokens, hkv, d, dtype, order", [
    (1900, 2, 64, BF16, "blocks"), (2500, 1, 128, F32, "requests"), (5000, 2, 64, BF16, "requests"),
    (5000, 1, 64, F32, "blocks"), (7000, 3, 128, BF16, "requests"), (9728, 1, 64, BF16, "blocks"),
    (10001, 1, 64, F32, "duplicates"), (6000, 2, 128, BF16, "shuffled"), (5500, 1, 64, BF16, "reversed")])
def test_gather(tokens, hkv, d, dtype, order):
    """Runs of every length, padding inside and between them, slots past the pool; rows of other
    tokens and heads as they were."""
    pkv = _pkv()
    rng = np.random.default_rng(tokens + hkv)
    nb = tokens // 16 + 12
    pools = _pools(rng, nb, hkv, d)
    slots = _slots(rng, order, tokens, nb, int(rng.integers(1, 16)))
    slots[rng.integers(0, tokens, 40)] = -1
    slots[700:733] = -5
    past = np.r_[40:56, rng.integers(60, tokens, 5)]    # (a whole block past the pool, and single slots)
    slots[past] = np.r_[nb * 16:nb * 16 + 16, nb * 16 + np.array([0, 1, 17, 1 << 36, 1 << 40])]
    wide = [torch.full((tokens, hkv + 1, d), 7.0, dtype=dtype, device="cuda") for _ in "kv"]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kc, vc = (torch.from_numpy(p).cuda() for p in pools)
    pkv.gather_cache_fp8(kc, vc, torch.from_numpy(slots).cuda(), *(w[:, :hkv] for w in wide), error_word=err)
    assert int(err) == pkv.ERR_SLOT
    for w, pool, key in zip(wide, pools, (True, False)):
        want = fp8.read_rows(pool, np.clip(slots, 0, nb * 16 - 1), hkv, d, key)
        want[slots < 0], want[slots >= nb * 16] = 7.0, 0.0
        assert np.array_equal(w[:, :hkv].double().cpu().numpy(), want, equal_nan=True)
        assert (w[:, hkv:] == 7).all()
