"""The 8-bit prefill of requests whose keys and values are converted ahead, and where the room
for that ends."""

import numpy as np
import pytest
import torch

from tests.fp8_support import Step, check
from tests.test_gpu_fp8_attention import rising_over_the_largest_values

pytestmark = pytest.mark.gpu


def _tile_bytes(hkv, d):
    return hkv * (2 * 256 * d + 4 * d + 4)


def _run(step, workspace=None, images=True, **kw):
    """(out, error word); `images`: whether some were made, which the workspace shows."""
    import paged_kv_cache_36_gb300 as pkv
    step.upload()
    ws = workspace
    if ws is None:
        ws = torch.zeros_like(pkv.new_workspace_fp8(step.H, step.hkv, step.d))
    out = pkv.paged_attention_varlen_fp8(*step.args(), workspace=ws, **kw)
    if workspace is None:
        tile = _tile_bytes(step.hkv, step.d)
        assert bool(ws[ws.numel() - (256 << 20) // tile * tile:][:1 << 16].any()) == images
    return out, pkv.read_error_word(ws)


@pytest.mark.parametrize("heads, hkv, d", [(8, 2, 128), (4, 4, 64), (7, 1, 128), (16, 1, 64), (10, 2, 64)])
def test_parity(heads, hkv, d):
    """Beside rows without images and decode rows; odd lengths, ends inside blocks and tiles."""
    more = 0 if d == 128 else 2000
    reqs = [(1, 50), (600, 500 + more), (33, 40), (5, 2000), (700, 403 + more), (0, 900), (130, 1500 + more), (1, 3)]
    step = Step(heads + d, reqs, heads, hkv, d, table_pad=2, stride_pad=1)
    out, err = _run(step)
    assert err == 0
    check(out, *step.reference())


@pytest.mark.parametrize("reqs, images", [([(4, 2500)], True), ([(4, 600)], False), ([(4, 1200)] * 60, False),
                                          ([(4, 600), (500, 700)], True), ([(900, 0)], True), ([(700, 0)], False)])
def test_which_requests_have_them(reqs, images):
    """Few query tiles: of long requests, unless there are many.  Many: where a CTA has enough (0.9 of
    its key tiles, 8 for 900 tokens, above 6.5 + 0.014 for each there is, of each KV head; without
    the 6.5 where the table and the tokens could be worth it: 60 of 10 key tiles are not)."""
    step = Step(len(reqs), reqs, 8, 2, 128)
    out, err = _run(step, images=images)
    assert err == 0
    check(out, *step.reference())


@pytest.mark.parametrize("scale", [-0.2, 5.0])
def test_scale(scale):
    step = Step(3, [(520, 700)], 4, 1, 128)
    step.scale = scale
    out, err = _run(step)
    assert err == 0
    check(out, *step.reference())


def test_nan():
    """In keys and values of a request with images, early, in the middle and in the last
    tokens, of either KV head and both halves of the dimensions."""
    step = Step(12, [(530, 600), (520, 600)], 4, 2, 128)
    for pos, h, dim in ((900, 0, 3), (901, 0, 100), (1129, 0, 64), (1000, 1, 127), (10, 1, 40), (900, 0, 4)):
        step.set(step.v, False, 0, pos, h, dim, 0xFF)
    step.set(step.k, True, 0, 1050, 1, 77, 0x7F)
    ref, tol = step.reference()
    assert ref[:530].isnan().any() and ref[530:].isfinite().all()
    out, err = _run(step)
    assert err == 0
    check(out, ref, tol)


@pytest.mark.parametrize("tiles", [0, 9, 20, 27])
def test_a_shorter_workspace(tiles):
    """Room for some of the requests' key tiles (9, 10 and 8 of them): the others are converted
    as they are needed, with the same result."""
    import paged_kv_cache_36_gb300 as pkv
    step = Step(5, [(520, 600), (600, 611), (1, 77), (530, 490)], 8, 2, 128)
    ws = pkv.new_workspace_fp8(8, 2, 128)
    whole, err = _run(step, ws)
    tile = _tile_bytes(2, 128)
    need = ws.numel() - (256 << 20) // tile * tile
    got, err = _run(step, ws[:need + tiles * tile])
    assert err == 0 and torch.equal(got, whole)
    check(got, *step.reference())
    with pytest.raises(pkv.PkvError, match="PKV_E_WORKSPACE"):
        pkv.paged_attention_varlen_fp8(*step.args(), workspace=ws[:need - 16])


def test_block_ids_outside_the_pool_read_as_zeros():
    import paged_kv_cache_36_gb300 as pkv
    step = Step(6, [(520, 700), (1, 5)], 4, 2, 128)
    blk = step.table[0, 40]
    step.k[blk] = step.v[blk] = 0
    ref, tol = step.reference()
    step.table[0, 40] = len(step.k)
    out, err = _run(step)
    assert err == pkv.ERR_BLOCK_ID
    check(out, ref, tol)


def test_a_workspace_used_again():
    """Other batches between two calls: nothing of the images stays."""
    import paged_kv_cache_36_gb300 as pkv
    ws = pkv.new_workspace_fp8(8, 2, 128)
    a = Step(1, [(520, 600), (40, 3)], 8, 2, 128)
    b = Step(2, [(300, 0), (1, 900), (800, 400)], 8, 2, 128)
    b.set(b.v, False, 2, np.arange(500, 700)[:, None], 0, np.arange(128), 0x7F)
    first, _ = _run(a, ws)
    second, _ = _run(b, ws)
    again, err = _run(a, ws)
    assert err == 0 and torch.equal(first, again) and first.isfinite().all()
    check(second, *b.reference())


def test_many_requests():
    """More requests than a plan in shared memory has entries, one of them with images."""
    reqs = [(2, i % 5) for i in range(4500)] + [(520, 600)] + [(1, 9)] * 300
    step = Step(8, reqs, 2, 1, 128)
    out, err = _run(step)
    assert err == 0
    check(out, *step.reference())


@pytest.mark.parametrize("room", [True, False])
@pytest.mark.parametrize("heads, hkv, d, more", [(8, 2, 128, 0), (4, 1, 64, 0), (4, 1, 64, 1000)])
def test_scores_that_rise(heads, hkv, d, more, room):
    """Scores of a key tile together 16 to 336 above the one before, or below it, in all rows,
    in some of a tile's and in a tile's half: the weights' reference moves, from weights that
    float32 holds and from others."""
    import paged_kv_cache_36_gb300 as pkv
    step = Step(heads + d, [(520, 800 + more), (300, 900 + more)], heads, hkv, d)
    step.scale = 1.0
    step.q.fill_(1.0)
    step.q[::3] = 0.5            # (rows that rise by half as much)
    step.q[5::7] = -1.0          # (and that fall)
    codes = {0: 0x00, 16: None, 40: None, 24: None, 240: None, 576: None}
    value = lambda c: next(x for x in range(0x7F) if (x & 7 | (8 if x >> 3 else 0)) * 2.0 ** (max(x >> 3, 1) - 10) == c / d)  # noqa: E731
    for c in codes:
        codes[c] = value(c)
    rises = [0, 16, 40, 24, 24, 240, 40, 240, 576, 576, 240]
    for r in range(2):
        n = step.seq[r]
        for h in range(hkv):
            for b in range(-(-n // 16)):
                step.set_scale(step.k, r, b, h, 127)
            for pos in range(n):
                c = rises[min(pos // 128, len(rises) - 1)]
                if pos % 128 >= 64 and pos // 128 == 3:
                    c = 40               # one half of a tile alone
                step.set(step.k, True, r, pos, h, np.arange(d), codes[c])
            step.set(step.k, True, r, np.arange(n), h, 7, step.rng.integers(0, 0x39, n).astype(np.uint8))
    ws = None
    if not room:
        ws = torch.zeros_like(pkv.new_workspace_fp8(heads, hkv, d))
        tile = _tile_bytes(hkv, d)
        ws = ws[:ws.numel() - (256 << 20) // tile * tile]
    # (11 key tiles of head_dim 64 are not worth the kernels)
    out, err = _run(step, ws, images=d == 128 or more > 0)
    assert err == 0
    check(out, *step.reference())


@pytest.mark.parametrize("room", [True, False])
@pytest.mark.parametrize("heads, hkv, d, mixed", [(4, 2, 128, False), (8, 2, 128, True), (4, 1, 64, True)])
def test_scores_that_rise_over_the_largest_values(heads, hkv, d, mixed, room):
    """Of requests over images and without (and of one that has no such values, beside them)."""
    import paged_kv_cache_36_gb300 as pkv
    more = 0 if d == 128 else 2000
    reqs = [(520, 800 + more), (300, 900 + more), (3, 700), (1, 500)]
    step = rising_over_the_largest_values(reqs, heads, hkv, d, mixed, seed=int(room))
    n = step.seq[1]
    for h in range(hkv):
        step.set(step.v, False, 1, np.arange(n)[:, None], h, np.arange(d),
                 step.rng.integers(0, 0x7F, (n, d)).astype(np.uint8))
        for b in range(-(-n // 16)):
            step.set_scale(step.v, 1, b, h, 120)
    ws = None
    if not room:
        ws = torch.zeros_like(pkv.new_workspace_fp8(heads, hkv, d))
        tile = _tile_bytes(hkv, d)
        ws = ws[:ws.numel() - (256 << 20) // tile * tile]
    out, err = _run(step, ws)
    assert err == 0
    ref, tol = step.reference()
    assert 1e38 < ref.abs().max() < 3e38
    check(out, ref, tol)


@pytest.mark.parametrize("heads, hkv, d", [(32, 2, 64), (16, 1, 128)])
def test_nan_of_one_query_tile_after_the_other(heads, hkv, d):
    """Without room for images, ten and more query tiles a CTA: NaN that some rows of a tile see, in
    some tiles, in several of a CTA in a row, and none in those between."""
    import paged_kv_cache_36_gb300 as pkv
    R = 160 // hkv + 40
    rng = np.random.default_rng(d)
    reqs = [(int(rng.integers(50, 65)) * 2 // hkv, int(rng.integers(0, 200))) for _ in range(R)]
    tpt = 128 // (heads // hkv)
    tiles = sum(-(-n // tpt) for n, _ in reqs) * hkv
    assert tiles > 1600
    step = Step(d, reqs, heads, hkv, d)
    for r, (n, past) in enumerate(reqs):
        if r // 7 % 3 == 0:     # (clean requests side by side)
            continue
        for pos in range(past, past + n, int(rng.integers(3, 20))):
            step.set(step.v, False, r, pos, int(rng.integers(hkv)), int(rng.integers(d)), 0x7F if pos % 2 else 0xFF)
    ref, tol = step.reference()
    seen = ref.isnan().any(-1)
    assert 0.05 < seen.double().mean() < 0.95
    ws = torch.zeros_like(pkv.new_workspace_fp8(heads, hkv, d))
    tile = _tile_bytes(hkv, d)
    out, err = _run(step, ws[:ws.numel() - (256 << 20) // tile * tile])
    assert err == 0
    check(out, ref, tol)
