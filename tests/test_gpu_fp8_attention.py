"""GPU parity of the attention over the 8-bit paged cache, within the bound derived in
tests/fp8_support.py."""

import numpy as np
import pytest
import torch

from oracle import fp8
from tests.fp8_support import Step, check

pytestmark = pytest.mark.gpu


def _pkv():
    import paged_kv_cache_36_gb300 as pkv
    return pkv


def _run(step, **kw):
    pkv = _pkv()
    step.upload()
    ws = pkv.new_workspace_fp8(step.H, step.hkv, step.d)
    out = pkv.paged_attention_varlen_fp8(*step.args(), workspace=ws, **kw)
    assert pkv.read_error_word(ws) == 0
    return out


HEADS = [(8, 2, 64), (32, 8, 128), (4, 4, 128), (7, 1, 64), (16, 1, 128), (15, 3, 128), (10, 5, 64), (18, 2, 64),
         (24, 12, 128), (34, 17, 64)]


@pytest.mark.parametrize("heads, hkv, d", HEADS)
def test_decode(heads, hkv, d):
    reqs = [(1, p) for p in (0, 1, 14, 15, 16, 17, 31, 32, 33, 63, 200, 511, 1000)]
    step = Step(heads + d, reqs, heads, hkv, d, table_pad=3, stride_pad=2)
    for hint in (1, 0):
        check(_run(step, max_query_len=hint), *step.reference())


@pytest.mark.parametrize("heads, hkv, d", HEADS)
def test_prefill(heads, hkv, d):
    reqs = [(2, 0), (5, 3), (17, 0), (0, 9), (40, 100), (130, 1), (3, 500)]
    step = Step(heads * 3 + d, reqs, heads, hkv, d, table_pad=1)
    check(_run(step), *step.reference())


@pytest.mark.parametrize("heads, hkv, d", [(32, 8, 128), (16, 4, 64), (6, 1, 128)])
def test_mixed(heads, hkv, d):
    reqs = [(1, 40), (33, 7), (1, 0), (0, 5), (1, 700), (300, 20), (1, 15), (2, 2000)]
    step = Step(heads + 1, reqs, heads, hkv, d)
    check(_run(step, max_query_len=300), *step.reference())


@pytest.mark.parametrize("reqs", [[(1, 30000)], [(1, 9000), (1, 3)], [(1, 2)] * 300, [(1, 100 + 7 * i) for i in range(80)],
                                  [(700, 0)], [(257, 1500)], [(2, 5000), (9, 3000)]])
def test_lengths(reqs):
    step = Step(len(reqs) + reqs[0][1], reqs, 8, 2, 128)
    check(_run(step, max_query_len=max(n for n, _ in reqs)), *step.reference())


@pytest.mark.parametrize("lo, hi", [(-117, -100), (-30, 30), (80, 110)])
@pytest.mark.parametrize("which", ["keys", "values"])
def test_scales_far_apart(lo, hi, which):
    """Block scales over the type's range.  Keys: with queries that keep the scores ordinary
    where they can, the softmax picks the loudest blocks.  Values: weight times value, whichever."""
    step = Step(lo + 200, [(1, 400), (40, 200)], 8, 2, 64)
    for pool, key in ((step.k, True), (step.v, False)):
        if (which == "keys") == key:
            p = pool.reshape(len(pool), 2, -1)
            p[:, :, 16 * 64] = step.rng.integers(127 + lo, 128 + hi, p.shape[:2])
    if which == "keys":
        step.q *= 2.0 ** -(hi + 6)
    check(_run(step), *step.reference())


@pytest.mark.parametrize("q_exp, lo, hi, scale_exp, prefill", [
    (120, -9, -5, -124, False),    # query times K's scale past 2^111, where the scores are ordinary
    (50, 80, 84, -143, False), (10, 115, 119, -138, False), (100, -20, -9, -100, True),
    (-120, -9, -5, 116, True),     # below 2^-126
    (-60, -80, -74, 125, False), (-100, -30, -24, 115, True)])
def test_exponents_that_cancel(q_exp, lo, hi, scale_exp, prefill):
    """Queries, K's scales and the softmax's scale far from 1, their product not: scores of a few
    units in single rows, and in those of several tokens too where <q, k> itself is a float32."""
    step = Step(300 + q_exp, [(1, 400), (1, 33)] + [(20, 100)] * prefill, 8, 2, 64)
    k = step.k.reshape(len(step.k), 2, -1)
    k[:, :, 16 * 64] = step.rng.integers(127 + lo, 128 + hi, k.shape[:2])
    step.q *= 2.0 ** q_exp
    step.scale = 2.0 ** scale_exp
    ref, tol = step.reference()
    assert step.q.isfinite().all() and (tol <= 2.0 ** -5 * ref.abs().max()).all()
    check(_run(step), ref, tol)


def test_unlikely_keys_with_large_values():
    """A key e^-60 as likely as the others holds the only values that are not zero."""
    step = Step(3, [(1, 299), (40, 260)], 4, 2, 128)
    step.scale = 1.0
    step.q.fill_(1.0)
    for r in range(2):
        for h in range(2):
            n = step.seq[r]
            step.set(step.k, True, r, np.arange(n)[:, None], h, np.arange(128), 0)
            step.set(step.v, False, r, np.arange(n)[:, None], h, np.arange(128), 0)
            step.set(step.k, True, r, 37, h, np.arange(60), 0xB8)          # -1 each, sixty of them
            step.set(step.v, False, r, 37, h, np.arange(128), 0x7E)
            for b in range(-(-n // 16)):
                step.set_scale(step.k, r, b, h, 127)
                step.set_scale(step.v, r, b, h, 200 if b == 2 else 127)
    check(_run(step), *step.reference())


def test_the_largest_values():
    """All values 1.75 2^127 or their negative, flat scores: sums stay finite, and so does the result."""
    step = Step(5, [(1, 3000), (1, 20), (300, 800), (40, 3)], 4, 2, 64)
    step.q *= 2.0 ** -12
    for pool, key in ((step.v, False),):
        for r in range(4):
            n = step.seq[r]
            step.set(pool, key, r, np.arange(n)[:, None], 0, np.arange(64), 0x7E)
            step.set(pool, key, r, np.arange(n)[:, None], 1, np.arange(64), 0xFE)
            for b in range(-(-n // 16)):
                for h in range(2):
                    step.set_scale(pool, r, b, h, 246)
    ref, tol = step.reference()
    assert ref.abs().max() < 3e38
    check(_run(step), ref, tol)


def test_the_largest_values_in_more_than_a_thousand_ranges():
    """Flat scores over 120000 keys of one KV head: ranges join to a finite result."""
    step = Step(6, [(1, 119999)], 2, 1, 64)
    step.q *= 2.0 ** -12
    n = step.seq[0]
    step.set(step.v, False, 0, np.arange(n)[:, None], 0, np.arange(64), 0x7E)
    step.v[:, 16 * 64] = 246
    ref, tol = step.reference()
    assert 2.9e38 < ref.abs().min() and ref.abs().max() < 3e38
    check(_run(step, max_query_len=1), ref, tol)


def rising_over_the_largest_values(reqs, heads, hkv, d, mixed, seed=0):
    """Scores that rise by 16 to 24 (2^23 to 2^35) every so many keys of a request, in halves of
    blocks too, and fall again; values 1.75 2^127 (of odd KV heads the negative), or where mixed
    some blocks of them between ordinary ones."""
    step = Step(seed + heads + d, reqs, heads, hkv, d)
    step.scale = 1.0
    step.q.fill_(1.0)
    scores = {0: 0x00, 16: 0x58, 18: 0x59, 36: 0x61, 40: 0x62, 56: 0x66, 72: 0x69, 80: 0x6A}
    rises = [0, 18, 18, 36, 56, 72, 40, 80, 16, 0]
    for r, n in enumerate(step.seq):
        each = max(n // 9, 8)
        for h in range(hkv):
            step.set(step.k, True, r, np.arange(n)[:, None], h, np.arange(d), 0)
            for i in range(0, n, each):
                step.set(step.k, True, r, np.arange(i, min(n, i + each)), h, 5, scores[rises[i // each % 10]])
            for b in range(-(-n // 16)):
                step.set_scale(step.k, r, b, h, 127)
                if not mixed or b % 3 == 1:
                    at = np.arange(16 * b, min(n, 16 * b + 16))
                    step.set(step.v, False, r, at[:, None], h, np.arange(d), 0xFE if h % 2 else 0x7E)
                    step.set_scale(step.v, r, b, h, 246)
    return step


@pytest.mark.parametrize("heads, hkv, d, mixed", [(4, 2, 64, False), (8, 2, 128, True), (16, 1, 64, True)])
def test_decode_of_scores_that_rise_over_the_largest_values(heads, hkv, d, mixed):
    step = rising_over_the_largest_values([(1, 3000), (1, 100), (1, 39), (1, 700)], heads, hkv, d, mixed)
    ref, tol = step.reference()
    assert 1e38 < ref.abs().max() < 3e38
    check(_run(step, max_query_len=1), ref, tol)


def test_nan_counts_for_the_rows_that_see_it():
    """NaN in a key or a value at a position makes what sees it NaN: of a value one dimension
    of the rows behind, of a key all of them."""
    step = Step(9, [(1, 100), (50, 90), (200, 0), (1, 33)], 8, 2, 64)
    step.set(step.v, False, 0, 60, 1, 5, 0x7F)
    step.set(step.v, False, 1, 120, 0, 63, 0xFF)      # seen by the rows from position 120 on
    step.set(step.v, False, 1, 10, 1, 0, 0x7F)        # by every row
    step.set(step.v, False, 2, 130, 1, 17, 0x7F)
    step.set(step.k, True, 2, 150, 0, 8, 0xFF)
    step.set(step.k, True, 3, 33, 1, 8, 0x7F)
    ref, tol = step.reference()
    assert ref.isnan().any() and ref.isfinite().any()
    for h in (0, 4):        # a key: every dimension of the rows behind it
        assert ref[51 + 150:251, 0].isnan().all()
    check(_run(step), ref, tol)


def test_scores_at_the_ends():
    """Large scores, a negative and a zero scale."""
    for scale in (40.0, -0.3, 0.0):
        step = Step(11, [(1, 200), (70, 65)], 8, 4, 128)
        step.scale = scale
        check(_run(step), *step.reference())


@pytest.mark.parametrize("scale", [0.0, 2.0 ** -149, -2.0 ** -130, 2.0 ** -126])
def test_the_smallest_scales_over_the_largest_sums(scale):
    """<q, k> up to 2^127 or near, in single rows and in those of several tokens: scores of a few units
    at most, of none at all with a scale of zero."""
    step = Step(12, [(1, 200), (70, 65), (3, 0)], 8, 4, 128, lo=0, hi=0)
    step.q.fill_(2.0 ** 114)
    step.q[::2] *= -1
    step.scale = scale
    ref, tol = step.reference()
    k = step.history(1)[0].sum(-1).abs().max() * 2.0 ** 114
    assert 2.0 ** 125 < k < 2.0 ** 127 and (tol <= 2.0 ** -5 * ref.abs().max()).all()
    check(_run(step), ref, tol)


def test_rows_left_alone_and_bad_metadata():
    pkv = _pkv()
    step = Step(4, [(1, 20), (1, 40), (6, 3), (7, 40), (1, 9)], 4, 2, 64).upload()
    ref, tol = step.reference()
    q = torch.cat([step.dq, torch.zeros(5, 4, 64, dtype=torch.bfloat16, device="cuda")])
    out = torch.full_like(q, 3.0)
    ws = pkv.new_workspace_fp8(4, 2, 64)
    step.dseq[1] += 1
    step.dpast[3] -= 50
    args = (q,) + step.args()[1:]
    pkv.paged_attention_varlen_fp8(*args, out=out, workspace=ws)
    assert pkv.read_error_word(ws) == pkv.ERR_METADATA
    good = [0, 2, 3, 4, 5, 6, 7, 15]
    check(out[:16], ref, tol, good)
    rest = torch.ones(21, dtype=torch.bool)
    rest[good] = False
    assert (out[rest.cuda()] == 3).all()


@pytest.mark.parametrize("bad", [-1, 10 ** 6])
def test_block_ids_outside_the_pool_read_as_zeros(bad):
    pkv = _pkv()
    step = Step(6, [(1, 100), (40, 60)], 4, 2, 64)
    for r, b in ((0, 2), (1, 0)):
        blk = step.table[r, b]
        step.k[blk] = step.v[blk] = 0
    ref, tol = step.reference()
    step.table[0, 2] = step.table[1, 0] = bad
    step.upload()
    ws = pkv.new_workspace_fp8(4, 2, 64)
    out = pkv.paged_attention_varlen_fp8(*step.args(), workspace=ws)
    assert pkv.read_error_word(ws) == pkv.ERR_BLOCK_ID
    check(out, ref, tol)


def test_same_bits_again_and_on_another_stream():
    pkv = _pkv()
    step = Step(8, [(1, 3000), (1, 77), (90, 1000)], 32, 8, 128).upload()
    a = pkv.paged_attention_varlen_fp8(*step.args())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = pkv.paged_attention_varlen_fp8(*step.args(), stream=s)
    s.synchronize()
    assert torch.equal(a, b)


def test_captured_steps():
    """Table, RoPE with the write, metadata and attention of a step in a graph, replayed with
    new inputs and lengths, against the same calls made eagerly."""
    pkv = _pkv()
    H, hkv, d, R, dev = 8, 2, 64, 3, "cuda"
    i32 = dict(dtype=torch.int32, device=dev)
    table = pkv.build_cos_sin_cache(4096, d, scaling="yarn", factor=4.0, original_max_position=1024)

    def state():
        return dict(kv=pkv.new_cache_fp8(64, hkv, d), ring=torch.arange(64, **i32), word=torch.zeros(1, **i32),
                    fs=torch.tensor([0, 64, 0, 0], device=dev), bt=torch.full((R, 24), -1, **i32),
                    new=torch.zeros(R, **i32), held=torch.zeros(R, **i32), ws=pkv.new_workspace_fp8(H, hkv, d),
                    rows=torch.zeros(48, H + 2 * hkv, d, dtype=torch.bfloat16, device=dev),
                    q=torch.zeros(48, H, d, dtype=torch.bfloat16, device=dev),
                    out=torch.zeros(48, H, d, dtype=torch.bfloat16, device=dev))

    def step(s):
        qsl, seq, slots, pos = pkv.build_step_metadata(s["new"], s["held"], s["bt"], s["ring"], s["fs"], 48,
                                                       error_word=s["word"])
        q, k, v = s["rows"][:, :H], s["rows"][:, H:H + hkv], s["rows"][:, H + hkv:]
        pkv.rope_reshape_and_cache_fp8(pos, q, k, v, *s["kv"], slots, table, query_out=s["q"], error_word=s["word"])
        pkv.paged_attention_varlen_fp8(s["q"], *s["kv"], s["bt"], qsl, seq, s["held"], d ** -0.5, out=s["out"],
                                       workspace=s["ws"])

    eager, graphed = state(), state()
    warm = state()
    warm["new"].fill_(3)
    step(warm)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(graphed)
    gen = torch.Generator(device=dev).manual_seed(0)
    held = [0, 0, 0]
    for new in ([20, 1, 0], [1, 17, 30], [1, 1, 1], [0, 2, 40]):
        rows = torch.randn(48, H + 2 * hkv, d, generator=gen, device=dev).to(torch.bfloat16)
        for s in (eager, graphed):
            s["rows"].copy_(rows)
            s["new"].copy_(torch.tensor(new))
            s["held"].copy_(torch.tensor(held))
        step(eager)
        g.replay()
        torch.cuda.synchronize()
        n = sum(new)
        assert torch.equal(eager["out"][:n], graphed["out"][:n]) and eager["out"][:n].isfinite().all()
        for a, b in zip(eager["kv"], graphed["kv"]):
            assert torch.equal(a, b)
        held = [a + b for a, b in zip(held, new)]
    assert int(eager["word"]) == int(graphed["word"]) == 0 == pkv.read_error_word(graphed["ws"])
    # and the last step's attention against float64 over what the cache holds
    r, n = 2, held[2]
    at = eager["bt"][r, torch.arange(n, device=dev) // 16].long() * 16 + torch.arange(n, device=dev) % 16
    k, v = (torch.empty(n, hkv, d, device=dev) for _ in "kv")
    pkv.gather_cache_fp8(*eager["kv"], at, k, v)
    q = eager["q"][2:42].double()
    for h in range(H):
        s = q[:, h] @ k[:, h // 4].double().T * d ** -0.5
        s = s.masked_fill(torch.arange(n, device=dev) > n - 40 + torch.arange(40, device=dev)[:, None], -torch.inf)
        want = torch.softmax(s, -1) @ v[:, h // 4].double()
        assert ((eager["out"][2:42, h].double() - want).abs() <= 2.0 ** -6 * v.abs().amax()).all()


def test_pools_past_two_to_the_32_bytes():
    """The blocks of a request at the far end of a pool of more than 2^32 bytes."""
    pkv = _pkv()
    step = Step(2, [(1, 50), (30, 20)], 8, 2, 128)
    ref, tol = step.reference()
    step.upload()
    nb, size = len(step.k), step.k.shape[1]
    far = (1 << 32) // size + 100
    kc, vc = (torch.zeros(far + nb, size, dtype=torch.uint8, device="cuda") for _ in "kv")
    kc[far:], vc[far:] = step.kc, step.vc
    bt = torch.where(step.bt >= 0, step.bt + far, -1).to(torch.int32)
    out = pkv.paged_attention_varlen_fp8(step.dq, kc, vc, bt, step.dqsl, step.dseq, step.dpast, step.scale)
    check(out, ref, tol)
    rows = torch.randn(3, 2, 128, device="cuda")
    slots = torch.tensor([(far + int(step.table[0, 0])) * 16 + 15, 0, (far + int(step.table[1, 0])) * 16], device="cuda")
    pkv.reshape_and_cache_fp8(rows, rows, kc, vc, slots)
    k, v = torch.empty_like(rows), torch.empty_like(rows)
    pkv.gather_cache_fp8(kc, vc, slots, k, v)
    # (the first slot's block holds other rows: its scale is 2^-5 at most, or what these need)
    assert ((k - rows).abs() <= rows.abs() * 2.0 ** -4 + 2.0 ** -12).all()
    assert ((v - rows).abs() <= rows.abs() * 2.0 ** -4 + 2.0 ** -12).all()
