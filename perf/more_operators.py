"""Cases, plain forms and 64-bit values of the operators of the 8-bit paged cache.

The operators: the table of rotary angles with its long-context scalings
(`build_cos_sin_cache`), the quantising cache write (`reshape_and_cache_fp8`), the
rotation fused with it (`rope_reshape_and_cache_fp8`), the read-back
(`gather_cache_fp8`) and attention over the 8-bit cache
(`paged_attention_varlen_fp8`: rows of one new token, and prefill chunks).

A cache is uint8 [num_blocks, Hkv * (16 D + 16)].  One block holds 16 tokens; KV head
h owns bytes [h (16 D + 16), (h + 1) (16 D + 16)): 16 D e4m3 codes, then the scale
byte e, then 15 zero bytes.  A value is code * 2^(e - 127), e clamped to [10, 246].
With P = D / 8, of token t and dimension d
  key code:    byte ((t / 8) (D / 64) + d / 64) 512 + (t % 8) 64 + d % 64
  value code:  byte (d % P) / 4 512 + ((d / P) 4 + (t % 8) / 2) 16 + (d % 4) 4 + (t / 8) 2 + t % 2
A call that writes row 0 of a block begins it anew (rows it does not write become
zero); else the scale only grows, and rows that stay are rounded to the new one.
"""

import math
import random

import numpy as np
import torch

own = False

BS = 16          # tokens per cache block
DEV = "cuda"


# --------------------------------------------------------------------- cases
def listed():
    return [
        # the table of a server that starts with a long context: some 131072 positions of a
        # whole head of 128, by parts (what repeats often stays, what is slow is stretched)
        dict(name="table_131072", op="table", rows=131072, start=0, rd=128, base=500000.0, scaling="parts",
             factor=8.0, length=8192, low=1.0, high=4.0, attention=1.0),
        # some rows behind a table of half a head, ramp over the pairs, with its attention factor: latency
        dict(name="table_more_rows", op="table", rows=1021, start=40000, rd=32, base=10000.0, scaling="yarn",
             factor=16.0, length=4096, low=1.0, high=32.0, attention=1.2772588722239782),
        # the new tokens of a 64-request decode step appended to blocks that hold others
        dict(name="write_decode64", op="write", reqs=64, new_lo=1, new_hi=1, past_hi=4096, hkv=8, d=128,
             dtype="bf16", fused=True, pad=0, shuffle=False, loud=False),
        # the largest prefill step of the serving trace (8192-token budget), K and V inside a
        # fused QKV projection's rows, some chunks beginning inside a block
        dict(name="write_8192", op="write", reqs=16, new_lo=512, new_hi=512, past_hi=2000, hkv=8, d=128,
             dtype="bf16", fused=True, pad=0, shuffle=False, loud=False),
        # an odd number of float32 rows read back, odd head count
        dict(name="read_f32_odd", op="read", tokens=7777, hkv=5, d=64, dtype="f32", pad=5),
        # RoPE and write of a 64-request decode step, half layout, whole head
        dict(name="rope_decode64", op="rope", reqs=64, new_lo=1, new_hi=1, past_hi=4096, heads=32, hkv=8, d=128,
             rd=128, neox=True, dtype="bf16", pad=0),
        # RoPE and write of the 8192-token prefill step, interleaved, half of each head
        dict(name="rope_8192", op="rope", reqs=16, new_lo=512, new_hi=512, past_hi=2000, heads=32, hkv=8, d=128,
             rd=64, neox=False, dtype="bf16", pad=0),
        # one request decodes alone: latency
        dict(name="decode_one", op="attend", decodes=1, ctx_lo=1000, ctx_hi=1000, prompts=0, q_lo=0, q_hi=0,
             past_hi=0, heads=8, hkv=2, d=64),
        # the decode step of 64 requests with contexts of 128 to 4096, Llama-3-8B heads
        dict(name="decode_batch64", op="attend", decodes=64, ctx_lo=128, ctx_hi=4096, prompts=0, q_lo=0,
             q_hi=0, past_hi=0, heads=32, hkv=8, d=128),
        # long-context decode: 8 requests of 131072 tokens, Llama-3-70B heads
        dict(name="decode_long", op="attend", decodes=8, ctx_lo=131072, ctx_hi=131072, prompts=0, q_lo=0,
             q_hi=0, past_hi=0, heads=64, hkv=8, d=128),
        # one whole prompt of 4096 tokens
        dict(name="prefill_4096", op="attend", decodes=0, ctx_lo=1, ctx_hi=1, prompts=1, q_lo=4096, q_hi=4096,
             past_hi=0, heads=32, hkv=8, d=128),
        # a 512-token chunk with history beside 256 decodes of 256 to 8192 tokens
        dict(name="mixed_step", op="attend", decodes=256, ctx_lo=256, ctx_hi=8192, prompts=1, q_lo=512,
             q_hi=512, past_hi=2048, heads=32, hkv=8, d=128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.499)))))))


def draw(rng):
    op = rng.choice(["table", "write", "write", "read", "rope", "rope", "decode", "decode", "prefill", "mixed"])
    if op == "table":
        rd = 4 * rng.randint(1, 32)
        rows = _log(rng, 1, 131072 * 128 // max(rd, 64))
        scaling = rng.choice(["none", "linear", "ntk", "parts", "yarn"])
        factor = round(math.exp(rng.uniform(0, math.log(64))), 3)
        low = rng.choice([1.0, 1.0, 0.5])
        return dict(op=op, rows=min(rows, 131072), start=rng.choice([0, 0, _log(rng, 1, 1 << 20)]), rd=rd,
                    base=rng.choice([10000.0, 500000.0, 1000000.0]), scaling=scaling, factor=factor,
                    length=_log(rng, 256, 32768), low=low, high=rng.choice([4.0, 32.0]),
                    attention=1.0 if scaling != "yarn" else 0.1 * math.log(factor) + 1.0)
    if op == "read":
        case = dict(op=op, tokens=_log(rng, 1, 16384), hkv=rng.choice([1, 2, 3, 4, 5, 8]), d=rng.choice([64, 128]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), pad=rng.choice([0, 0, 1, 7]))
        if case["dtype"] == "f32":
            case["tokens"] = max(1, case["tokens"] // 2)
        return case
    if op in ("write", "rope"):
        reqs = _log(rng, 1, 512)
        hi = _log(rng, 1, max(1, 8192 // reqs))
        d = rng.choice([64, 128])
        case = dict(op=op, reqs=reqs, new_lo=max(1, hi // rng.choice([1, 2, 16])), new_hi=hi,
                    past_hi=rng.choice([0, 15, 400, 2000]), hkv=rng.choice([1, 2, 3, 4, 5, 8]), d=d,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), pad=rng.choice([0, 0, 1, 7]))
        if case["dtype"] == "f32":
            case["new_hi"] = max(1, hi // 2)
            case["new_lo"] = min(case["new_lo"], case["new_hi"])
        if op == "write":
            case.update(fused=rng.choice([True, False]), shuffle=rng.choice([True, False, False]),
                        loud=rng.choice([True, False]))
        else:
            case.update(heads=case["hkv"] * rng.choice([1, 2, 4, 4, 7, 8]), rd=rng.choice([d, d, d // 2, d // 4]),
                        neox=rng.choice([True, False]))
        return case
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 3, 4, 5, 8, 8])
    group = rng.choice([1, 2, 4, 4, 5, 6, 7, 8, 16] if hkv <= 4 else [1, 2, 4, 4, 5, 7, 8])
    case = dict(op="attend", decodes=0, ctx_lo=1, ctx_hi=1, prompts=0, q_lo=0, q_hi=0, past_hi=0,
                heads=hkv * group, hkv=hkv, d=d)
    if op in ("decode", "mixed"):
        n = _log(rng, 1, 256)
        hi = _log(rng, 1, min(131072, (1 << 20) // n) if op == "decode" else min(8192, (1 << 19) // n))
        case.update(decodes=n, ctx_lo=max(1, hi // rng.choice([1, 2, 32])), ctx_hi=hi)
    if op in ("prefill", "mixed"):
        n = rng.choice([1, 1, 2, 3, 4])
        hi = _log(rng, 2, 2048 // n)
        case.update(prompts=n, q_lo=max(0, hi // rng.choice([1, 2, 64])), q_hi=hi, past_hi=rng.choice([0, 0, 17, 1000, 2000]))
    return case


def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _lengths(case):
    """The case's own request lengths (host integers, the same for every seed): new tokens
    and tokens before them."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    if case["op"] in ("write", "rope"):
        past = [rng.randint(0, case["past_hi"]) for _ in range(case["reqs"])]
        return [rng.randint(case["new_lo"], case["new_hi"]) for _ in past], past
    q, past = [], []
    for _ in range(case["prompts"]):
        q.append(rng.randint(case["q_lo"], case["q_hi"]))
        past.append(rng.randint(case["past_hi"] // 2, case["past_hi"]))
    if q:
        q[0] = max(1, q[0])
    for _ in range(case["decodes"]):
        q.append(1)
        past.append(rng.randint(case["ctx_lo"], case["ctx_hi"]) - 1)
    return q, past


def _blocks(tokens):
    return -(-tokens // BS)


def work(case):
    op = case["op"]
    if op == "table":
        return {"bytes": 4 * case["rows"] * case["rd"], "flops": 0}
    es = 4 if case.get("dtype") == "f32" else 2
    row = 2 * case["hkv"] * case["d"]             # values of a token, K and V
    held = 2 * case["hkv"] * (case["d"] + 1)      # bytes of a token in the cache
    if op == "read":
        return {"bytes": case["tokens"] * (held + es * row + 8), "flops": 0}
    if op in ("write", "rope"):
        new, past = _lengths(case)
        t, stay = sum(new), sum(p % BS for p in past)
        # rows in, the cache written, and read back with the rows that stayed in the blocks
        n = t * (es * row + held + 8) + (t + stay) * (held + (es if op == "write" else 2) * row + 8)
        if op == "rope":
            n += t * (2 * es * case["heads"] * case["d"] + 4 * case["rd"] + 8)
        return {"bytes": n, "flops": 0}
    q, past = _lengths(case)
    ctx = sum(p + n for p, n in zip(past, q) if n)
    rows = sum(q)
    pairs = sum(n * p + n * (n + 1) // 2 for p, n in zip(past, q))
    return {"bytes": ctx * held + 2 * rows * case["heads"] * case["d"] * 2 + 4 * _blocks(ctx),
            "flops": 4 * pairs * case["heads"] * case["d"]}


# ------------------------------------------------- the cache, in torch operations
def _chunk(d):
    return BS * d + BS


def _power(e):
    """2^(e - 127) as float32, from its bits (e in [1, 254])."""
    return (e.int() << 23).view(torch.float32)


def _scale_of(amax):
    """The scale byte of rows whose largest finite magnitude is amax (float32)."""
    bits = amax.contiguous().view(torch.int32)
    return ((bits >> 23) - 8 + ((bits & 0x7fffff) > 0x600000)).clamp(10, 246)


def _round(y):
    """float32 to the e4m3 codes' values, to nearest even, 448 at most; NaN stays."""
    a = y.abs().clamp(max=448.0)                                        # (clamp keeps NaN)
    step = _power((a.contiguous().view(torch.int32) >> 23).clamp(121, 135) - 3)   # of its binade, 2^-9 at least
    return torch.copysign(torch.round(a / step) * step, y)


def _open(codes, d, is_key):
    """Code bytes [..., 16 D] -> a view [..., 16 tokens, D] (as split dimensions, transposed)."""
    if is_key:   # [t / 8][d / 64][t % 8][d % 64]
        c = codes.unflatten(-1, (2, d // 64, 8, 64))
        return c.transpose(-3, -2)                                       # [2, 8, D / 64, 64]
    c = codes.unflatten(-1, (d // 32, 8, 4, 4, 2, 2))                    # [(d % P) / 4][d / P][(t % 8) / 2][d % 4][t / 8][t % 2]
    n = c.dim() - 6
    return c.permute(*range(n), n + 4, n + 2, n + 5, n + 1, n, n + 3)    # [2, 4, 2, 8, P / 4, 4]


def _values_of(blocks, hkv, d, is_key):
    """uint8 [..., block bytes] -> float32 codes' values [..., Hkv, 16, D], scale bytes [..., Hkv]."""
    p = blocks.unflatten(-1, (hkv, _chunk(d)))
    c = _open(p[..., :BS * d], d, is_key)
    x = c.reshape(*p.shape[:-1], BS, d).view(torch.float8_e4m3fn).float()
    return x, p[..., BS * d].int().clamp(10, 246)


def _read(blocks, hkv, d, is_key):
    """uint8 [..., block bytes] -> float32 [..., 16 tokens, Hkv, D]."""
    x, e = _values_of(blocks, hkv, d, is_key)
    x *= _power(e)[..., None, None]
    return x.transpose(-3, -2)


def _write(pool, x, slots, d, is_key):
    """Rows x float32 [n, Hkv, D] to their slots of a pool, by the rule at the top."""
    hkv = x.shape[1]
    at, of = torch.unique(slots // BS, return_inverse=True)
    off = slots % BS
    old, e_old = _values_of(pool[at], hkv, d, is_key)
    anew = torch.zeros(len(at), dtype=torch.bool, device=x.device)
    anew[of[off == 0]] = True
    fine = torch.isfinite(x)
    amax = torch.where(fine, x, 0).abs().amax(-1)
    most = torch.zeros(len(at), hkv, device=x.device).scatter_reduce_(0, of[:, None].expand(-1, hkv), amax, "amax")
    e_old = torch.where(anew[:, None], 10, e_old)
    e = torch.maximum(_scale_of(most), e_old)
    # rows that stay, at the new scale (a power of two: exact down to the rounding; all of it below 2^-126)
    old = torch.where(anew[:, None, None, None], 0, _round(old * _power((e_old - e + 127).clamp(min=1))[..., None, None]))
    old[of, :, off] = _round(torch.where(fine, x, torch.nan) * _power(254 - e[of])[..., None])
    p = pool.view(pool.shape[0], hkv, _chunk(d))
    c = torch.empty(len(at), hkv, BS * d, dtype=torch.uint8, device=x.device)
    v = _open(c, d, is_key)
    v.copy_(old.to(torch.float8_e4m3fn).view(torch.uint8).view(v.shape))
    p[at, :, :BS * d] = c
    p[at, :, BS * d] = e.to(torch.uint8)


# --------------------------------------------------------------------- inputs
def _values(gen, tokens, hkv, d):
    """Rows as a K or V projection gives them: a scale per channel (a few loud
    ones), a scale per token."""
    g = dict(generator=gen, device=DEV)
    channel = torch.exp2(torch.randn(hkv, d, **g)) * torch.where(torch.rand(hkv, d, **g) < 0.02, 8.0, 0.5)
    x = torch.randn(tokens, hkv, d, **g)
    return x * channel * torch.exp2(0.5 * torch.randn(tokens, 1, 1, **g))


def _pool(gen, blocks, hkv, d):
    """Bytes that others left: any codes, scales as caches have them."""
    g = dict(generator=gen, device=DEV)
    pool = torch.randint(0, 256, (blocks, hkv * _chunk(d)), dtype=torch.uint8, **g)
    head = pool.view(blocks, hkv, _chunk(d))[..., BS * d:]
    head.zero_()
    head[..., 0] = torch.randint(115, 125, (blocks, hkv), dtype=torch.uint8, **g)
    return pool


def _spread(gen, new, past, spare):
    """A pool's size, and slots of every position of requests of past + new tokens."""
    g = dict(generator=gen, device=DEV)
    count = [_blocks(p + n) for p, n in zip(past, new)]
    nblk = sum(count) + spare
    ids = torch.randperm(nblk, **g)[:sum(count)]
    lens = torch.tensor([p + n for p, n in zip(past, new)], device=DEV)
    r = torch.repeat_interleave(torch.arange(len(new), device=DEV), lens)
    pos = torch.arange(len(r), device=DEV) - (torch.cumsum(lens, 0) - lens)[r]
    first = torch.tensor(np.concatenate([[0], np.cumsum(count)[:-1]]), device=DEV)
    return nblk, r, pos, ids[first[r] + pos // BS] * BS + pos % BS


def _padded(gen, x, pad):
    """int64 [n] with `pad` entries -1 among the last ones, and where they are."""
    if not pad:
        return x
    return torch.cat((x, torch.full((pad,), -1, dtype=x.dtype, device=DEV)))


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed * 7919 + 17)
    g = dict(generator=gen, device=DEV)
    op = case["op"]
    if op == "table":
        # (a table has no data but its numbers: another seed is another stretch of positions)
        return dict(case=case, start=case["start"] + seed % 64,
                    out=torch.empty(case["rows"], case["rd"], dtype=torch.float32, device=DEV))
    hkv, d = case["hkv"], case["d"]
    if op == "read":
        t, dt = case["tokens"], _dtype(case)
        nblk = _blocks(t) + 8
        kpool, vpool = _pool(gen, nblk, hkv, d), _pool(gen, nblk, hkv, d)
        order = torch.randperm(nblk * BS, **g)
        whole = torch.arange(nblk * BS, device=DEV)
        _write(kpool, _values(gen, nblk * BS, hkv, d), whole, d, True)
        _write(vpool, _values(gen, nblk * BS, hkv, d), whole, d, False)
        slots = order[:t].contiguous()
        if case["pad"]:
            slots[torch.randperm(t, **g)[:case["pad"]]] = -1
        return dict(case=case, kpool=kpool, vpool=vpool, back=slots,
                    kout=torch.zeros(t, hkv, d, dtype=dt, device=DEV), vout=torch.zeros(t, hkv, d, dtype=dt, device=DEV))
    if op in ("write", "rope"):
        dt = _dtype(case)
        new, past = _lengths(case)
        nblk, r, pos, slots = _spread(gen, new, past, 8)
        kpool, vpool = _pool(gen, nblk, hkv, d), _pool(gen, nblk, hkv, d)
        held = torch.tensor(past, device=DEV)[r]
        stay = (pos < held) & (pos >= held // BS * BS)    # in the block that gets the next token
        if bool(stay.any()):
            n = int(stay.sum())
            _write(kpool, _values(gen, n, hkv, d), slots[stay], d, True)
            _write(vpool, _values(gen, n, hkv, d), slots[stay], d, False)
        fresh = slots[pos >= held]
        positions = _padded(gen, pos[pos >= held], case["pad"]).clamp(min=0)
        fill = _padded(gen, fresh, case["pad"])
        if case.get("shuffle"):
            order = torch.randperm(len(fill), **g)
            fill, positions = fill[order], positions[order]
        t = len(fill)
        k, v = _values(gen, t, hkv, d), _values(gen, t, hkv, d)
        if case.get("loud"):    # tokens that outgrow the scale of the rows before them
            k *= torch.where(torch.rand(t, 1, 1, **g) < 0.1, 64.0, 1.0)
            v *= torch.where(torch.rand(t, 1, 1, **g) < 0.1, 64.0, 1.0)
        k, v = k.to(dt), v.to(dt)
        back = torch.cat((fresh, slots[stay]))
        s = dict(case=case, kpool=kpool, vpool=vpool, slots=fill.contiguous(), back=back.contiguous())
        if op == "write":
            if case["fused"]:   # [q heads | k heads | v heads] rows of one projection
                rows = torch.zeros(t, 6 * hkv, d, dtype=dt, device=DEV)
                rows[:, 4 * hkv:5 * hkv], rows[:, 5 * hkv:] = k, v
                k, v = rows[:, 4 * hkv:5 * hkv], rows[:, 5 * hkv:]
            out = dt
        else:
            h, rd = case["heads"], case["rd"]
            rows = torch.cat((torch.randn(t, h, d, **g).to(dt), k, v), 1)
            q, k, v = rows[:, :h], rows[:, h:h + hkv], rows[:, h + hkv:]
            most = int(max(p + n for p, n in zip(past, new)))
            inv = 10000.0 ** (-torch.arange(0, rd, 2, device=DEV, dtype=torch.float64) / rd)
            angle = torch.arange(most, device=DEV, dtype=torch.float64)[:, None] * inv
            s.update(q=q, qout=torch.empty(t, h, d, dtype=dt, device=DEV), positions=positions.contiguous(),
                     table=torch.cat((angle.cos(), angle.sin()), 1).float().contiguous())
            out = torch.bfloat16
        s.update(k=k, v=v, kout=torch.zeros(len(back), hkv, d, dtype=out, device=DEV),
                 vout=torch.zeros(len(back), hkv, d, dtype=out, device=DEV))
        return s
    q, past = _lengths(case)
    seq = [p + n for p, n in zip(past, q)]
    count = [_blocks(n) for n in seq]
    used = sum(count)
    nblk = used + used // 4 + 4
    # blocks scattered over the pool; what no token has written is left as it was: noise
    kpool, vpool = _pool(gen, nblk, hkv, d), _pool(gen, nblk, hkv, d)
    width = max(count + [1])
    table = torch.full((len(q), width), -1, dtype=torch.int32, device=DEV)
    col = torch.arange(width, device=DEV)
    table[col < torch.tensor(count, device=DEV).unsqueeze(1)] = torch.randperm(nblk, **g)[:used].to(torch.int32)
    lens = torch.tensor(seq, device=DEV)
    first = torch.cumsum(torch.tensor(count, device=DEV), 0) - torch.tensor(count, device=DEV)
    ends = torch.cumsum(torch.tensor(count, device=DEV), 0)
    for lo in range(0, used, 1 << 13):      # blocks, so that each is written once
        b = torch.arange(lo, min(used, lo + (1 << 13)), device=DEV)
        r = torch.searchsorted(ends, b, right=True)
        p = ((b - first[r]) * BS)[:, None] + torch.arange(BS, device=DEV)
        slots = (table[r, b - first[r]].long() * BS)[:, None] + torch.arange(BS, device=DEV)
        live = p < lens[r][:, None]
        slots = slots[live]
        _write(kpool, _values(gen, len(slots), hkv, d), slots, d, True)
        _write(vpool, _values(gen, len(slots), hkv, d), slots, d, False)
    i32 = dict(dtype=torch.int32, device=DEV)
    rows = sum(q)
    # codes of tokens behind a request's end are noise again (NaN among them)
    last = torch.tensor([i for i, n in enumerate(seq) if n % BS], dtype=torch.int64, device=DEV)
    if len(last):
        blk = table[last, torch.tensor([n // BS for n in seq if n % BS], device=DEV)].long()
        dead = torch.arange(BS, device=DEV) >= torch.tensor([n % BS for n in seq if n % BS], device=DEV)[:, None]
        for pool, is_key in ((kpool, True), (vpool, False)):
            c = pool[blk].unflatten(-1, (hkv, _chunk(d)))
            codes = c[..., :BS * d].contiguous()
            v = _open(codes, d, is_key)
            noise = torch.randint(0, 256, (len(blk), hkv, BS, d), dtype=torch.uint8, **g)
            flat = torch.where(dead[:, None, :, None], noise, v.reshape(noise.shape))
            v.copy_(flat.view(v.shape))
            c[..., :BS * d] = codes
            pool[blk] = c.flatten(-2)
    return dict(case=case, kpool=kpool, vpool=vpool, table=table,
                q=torch.randn(rows, case["heads"], d, **g).to(torch.bfloat16),
                out=torch.empty(rows, case["heads"], d, dtype=torch.bfloat16, device=DEV),
                qsl=torch.tensor(np.concatenate([[0], np.cumsum(q)]), **i32),
                seq=torch.tensor(seq, **i32), past=torch.tensor(past, **i32), longest=max(q), scale=d ** -0.5)


# ------------------------------------------------------------------ plain forms
def _plain_table(s):
    """In 64 bits: angles of far positions lose theirs in 32."""
    c = s["case"]
    rd, factor = c["rd"], c["factor"]
    i = torch.arange(rd // 2, dtype=torch.float64, device=DEV)
    base = c["base"] * factor ** (rd / (rd - 2)) if c["scaling"] == "ntk" else c["base"]
    inv = base ** (-2 * i / rd)
    if c["scaling"] == "linear":
        inv = inv / factor
    elif c["scaling"] in ("parts", "yarn"):
        if c["scaling"] == "parts":
            keep = ((c["length"] * inv / (2 * math.pi) - c["low"]) / (c["high"] - c["low"])).clamp(0, 1)
        else:
            def pair(turns):
                return rd * math.log(c["length"] / (2 * math.pi * turns)) / (2 * math.log(base))
            lo, hi = max(math.floor(pair(c["high"])), 0), min(math.ceil(pair(c["low"])), rd - 1)
            keep = 1 - ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        inv = inv * keep + inv / factor * (1 - keep)
    angle = torch.arange(s["start"], s["start"] + c["rows"], dtype=torch.float64, device=DEV)[:, None] * inv
    return (torch.cat((angle.cos(), angle.sin()), 1) * c["attention"]).float()


def _plain_read(s):
    c = s["case"]
    at = s["back"].clamp(min=0)
    got = []
    for pool, is_key, out in ((s["kpool"], True, s["kout"]), (s["vpool"], False, s["vout"])):
        x = _read(pool, c["hkv"], c["d"], is_key).flatten(0, 1)[at]
        got.append(torch.where((s["back"] >= 0)[:, None, None], x, 0).to(out.dtype))
    return got


def _rotate(x, s):
    """float32 [t, heads, D], each row by its position's angles."""
    rd, half = s["case"]["rd"], s["case"]["rd"] // 2
    at = s["table"][s["positions"]][:, None]
    cos, sin = at[..., :half], at[..., half:]
    if s["case"]["neox"]:
        a, b = x[..., :half], x[..., half:rd]
        return torch.cat((a * cos - b * sin, b * cos + a * sin, x[..., rd:]), -1)
    a, b = x[..., 0:rd:2], x[..., 1:rd:2]
    return torch.cat((torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2), x[..., rd:]), -1)


def _plain_write(s):
    d, live = s["case"]["d"], s["slots"] >= 0
    k = s["k"].float()
    if "q" in s:
        s["qout"].copy_(_rotate(s["q"].float(), s))
        k = _rotate(k, s)
    _write(s["kpool"], k[live], s["slots"][live], d, True)
    _write(s["vpool"], s["v"].float()[live], s["slots"][live], d, False)


def _plain_rows(s, lo, hi):
    """Requests [lo, hi) as one padded batch, written to their rows of out."""
    c = s["case"]
    if hi <= lo:
        return
    q_len = (s["qsl"][lo + 1:hi + 1] - s["qsl"][lo:hi]).long()
    most_q = s["longest"] if lo == 0 and c["prompts"] else 1
    u = torch.arange(most_q, device=DEV)
    row = (s["qsl"][lo:hi, None] + torch.minimum(u, (q_len - 1)[:, None])).clamp(min=0)
    q = s["q"][row].float().unflatten(2, (c["hkv"], -1)).permute(0, 2, 3, 1, 4)       # [R, Hkv, G, Q, D]
    group = q.shape[2]
    table = s["table"][lo:hi].clamp(min=0).long()
    k = _read(s["kpool"][table], c["hkv"], c["d"], True).flatten(1, 2).transpose(1, 2)
    v = _read(s["vpool"][table], c["hkv"], c["d"], False).flatten(1, 2).transpose(1, 2)
    j = torch.arange(k.shape[2], device=DEV)
    v.masked_fill_((j >= s["seq"][lo:hi, None])[:, None, :, None], 0)
    score = (q.flatten(2, 3) @ k.transpose(2, 3)).unflatten(2, (group, -1)) * s["scale"]
    seen = j <= (s["past"][lo:hi, None] + u)[:, :, None]
    score.masked_fill_(~seen[:, None, None], -torch.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    o = ((p.flatten(2, 3) @ v).unflatten(2, (group, -1)) / p.sum(-1, keepdim=True)).permute(0, 3, 1, 2, 4).flatten(2, 3)
    live = u < q_len[:, None]
    s["out"][row[live]] = o[live].to(s["out"].dtype)


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import paged_kv_cache_36_gb300 as pkv
        if op == "table":
            return pkv.build_cos_sin_cache(c["rows"], c["rd"], base=c["base"], scaling=c["scaling"], factor=c["factor"],
                                           original_max_position=c["length"], low=c["low"], high=c["high"],
                                           attention_factor=c["attention"], start=s["start"], out=s["out"])
        if op == "attend":
            if "workspace" not in s:   # kept from call to call, as a server keeps it
                s["workspace"] = pkv.new_workspace_fp8(c["heads"], c["hkv"], c["d"])
            return pkv.paged_attention_varlen_fp8(s["q"], s["kpool"], s["vpool"], s["table"], s["qsl"], s["seq"],
                                                  s["past"], s["scale"], out=s["out"], workspace=s["workspace"],
                                                  max_query_len=s["longest"])
        if op == "write":
            pkv.reshape_and_cache_fp8(s["k"], s["v"], s["kpool"], s["vpool"], s["slots"])
        elif op == "rope":
            pkv.rope_reshape_and_cache_fp8(s["positions"], s["q"], s["k"], s["v"], s["kpool"], s["vpool"], s["slots"],
                                           s["table"], is_neox=c["neox"], query_out=s["qout"])
        pkv.gather_cache_fp8(s["kpool"], s["vpool"], s["back"], s["kout"], s["vout"])
        return [s["kout"], s["vout"]] + ([s["qout"]] if op == "rope" else [])
    if op == "table":
        return _plain_table(s)
    if op == "attend":
        _plain_rows(s, 0, c["prompts"])
        _plain_rows(s, c["prompts"], c["prompts"] + c["decodes"])
        return s["out"]
    if op in ("write", "rope"):
        _plain_write(s)
    return _plain_read(s) + ([s["qout"]] if op == "rope" else [])


# ------------------------------------------------------------- 64-bit definition
def _grid64():
    """The magnitudes of e4m3, ascending (index: the code's low seven bits)."""
    return torch.tensor([m / 512 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127],
                        dtype=torch.float64, device=DEV)


def _power64(k):
    """2^k as float64 [n, 1, 1], from its bits."""
    return ((k + 1023) << 52).view(torch.float64)[:, None, None]


def _near64(y):
    """The grid's nearest to y (float64), of two equally near the one of even index; NaN for what is not finite."""
    grid = _grid64()
    hi = torch.searchsorted(grid, y.abs()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = (grid[hi] - y.abs()).abs(), (y.abs() - grid[lo]).abs()
    take = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return torch.where(torch.isfinite(y), torch.copysign(grid[take], y), torch.nan)


def _bytes64(d, is_key):
    """Where the codes of a head's 16 x D values are in its chunk."""
    t, i = torch.meshgrid(torch.arange(BS, device=DEV), torch.arange(d, device=DEV), indexing="ij")
    if is_key:
        return (t // 8 * (d // 64) + i // 64) * 512 + t % 8 * 64 + i % 64
    p = d // 8
    return i % p // 4 * 512 + (i // p * 4 + t % 8 // 2) * 16 + i % 4 * 4 + t // 8 * 2 + t % 2


def _codes64(pool, blk, h, d, is_key):
    """float64 [n, 16, D] of blocks blk, KV head h, and their scale exponents."""
    at = h * _chunk(d)
    code = pool[blk][:, at + _bytes64(d, is_key)].long()
    grid = torch.cat((_grid64(), torch.tensor([torch.nan], dtype=torch.float64, device=DEV)))
    x = torch.where(code >= 128, -grid[code % 128], grid[code % 128])
    return x, pool[blk, at + BS * d].long().clamp(10, 246) - 127


def _written64(pool, x, slots, back, d, is_key):
    """What the slots `back` hold after rows x (float64) went to `slots` (negative ones left out)."""
    live = slots >= 0
    x, slots = x[live], slots[live]
    at, of = torch.unique(slots // BS, return_inverse=True)
    off, n = slots % BS, len(at)
    got = []
    for h in range(x.shape[1]):
        old, e_old = _codes64(pool, at, h, d, is_key)
        rows = torch.zeros(n, BS, d, dtype=torch.float64, device=DEV)
        new = torch.zeros(n, BS, dtype=torch.bool, device=DEV)
        rows[of, off], new[of, off] = x[:, h], True
        amax = torch.where(torch.isfinite(rows), rows, 0).abs().amax((1, 2))
        m, ex = torch.frexp(amax)                                   # m in [1/2, 1): 448 = 7/8 2^9
        e = torch.where(amax > 0, (ex - 9 + (m > 0.875).int()).clamp(-117, 119), -117).long()
        e_old = torch.where(new[:, 0], -117, e_old)
        e = torch.maximum(e, e_old)
        stay = torch.where(new[:, :1, None], 0.0, _near64(old * _power64(e_old - e)))
        rows = torch.where(new[..., None], _near64(rows * _power64(-e)), stay) * _power64(e)
        got.append(rows[torch.searchsorted(at, back // BS), back % BS])
    return torch.stack(got, 1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "table":
        n, rd = case["rows"], case["rd"]
        out = np.empty((n, rd))
        p = np.arange(s["start"], s["start"] + n, dtype=np.float64)
        for i in range(rd // 2):
            f = math.exp(-2 * i / rd * math.log(case["base"]))
            if case["scaling"] == "linear":
                f /= case["factor"]
            elif case["scaling"] == "ntk":
                f = math.exp(-2 * i / rd * (math.log(case["base"]) + rd / (rd - 2) * math.log(case["factor"])))
            elif case["scaling"] == "parts":
                turns = case["length"] * f / (2 * math.pi)
                keep = min(1.0, max(0.0, (turns - case["low"]) / (case["high"] - case["low"])))
                f = keep * f + (1 - keep) * f / case["factor"]
            elif case["scaling"] == "yarn":
                ends = [rd / 2 * math.log(case["length"] / (2 * math.pi * x), case["base"]) for x in (case["high"], case["low"])]
                lo, hi = max(0, math.floor(ends[0])), min(rd - 1, math.ceil(ends[1]))
                slow = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
                f = (1 - slow) * f + slow * f / case["factor"]
            out[:, i], out[:, rd // 2 + i] = np.cos(p * f) * case["attention"], np.sin(p * f) * case["attention"]
        return out
    hkv, d = case["hkv"], case["d"]
    if op == "read":
        at = s["back"].clamp(min=0)
        got = []
        for pool, is_key in ((s["kpool"], True), (s["vpool"], False)):
            heads = []
            for h in range(hkv):
                x, e = _codes64(pool, torch.arange(len(pool), device=DEV), h, d, is_key)
                heads.append((x * _power64(e)).flatten(0, 1)[at])
            got.append(torch.where((s["back"] >= 0)[:, None, None], torch.stack(heads, 1), 0.0))
        return got
    if op in ("write", "rope"):
        k, q = s["k"].double(), None
        if op == "rope":
            rd = case["rd"]
            turn = torch.complex(s["table"][:, :rd // 2].double(), s["table"][:, rd // 2:].double())[s["positions"]][:, None]
            out = []
            for x in (k, s["q"].double()):
                y = x.clone()
                if case["neox"]:
                    z = torch.complex(x[..., :rd // 2].contiguous(), x[..., rd // 2:rd].contiguous()) * turn
                    y[..., :rd // 2], y[..., rd // 2:rd] = z.real, z.imag
                else:
                    z = torch.view_as_complex(x[..., :rd].contiguous().unflatten(-1, (-1, 2))) * turn
                    y[..., :rd] = torch.view_as_real(z).flatten(-2)
                out.append(y)
            k, q = out
        got = [_written64(s["kpool"], k, s["slots"], s["back"], d, True),
               _written64(s["vpool"], s["v"].double(), s["slots"], s["back"], d, False)]
        return got if q is None else got + [q]
    q_len, past = _lengths(case)
    group = case["heads"] // hkv
    out = torch.zeros(sum(q_len), case["heads"], d, dtype=torch.float64, device=DEV)
    row = 0
    for r, (n, p) in enumerate(zip(q_len, past)):
        if n == 0:
            continue
        blk = s["table"][r, :_blocks(p + n)].long()
        hide = torch.arange(p + n, device=DEV)[None, :] > p + torch.arange(n, device=DEV)[:, None]
        for g in range(hkv):
            k, ke = _codes64(s["kpool"], blk, g, d, True)
            v, ve = _codes64(s["vpool"], blk, g, d, False)
            k = (k * _power64(ke)).flatten(0, 1)[:p + n]
            v = (v * _power64(ve)).flatten(0, 1)[:p + n]
            for h in range(g * group, (g + 1) * group):
                a = s["q"][row:row + n, h].double() @ k.T * s["scale"]
                a = torch.softmax(a.masked_fill(hide, -torch.inf), -1)
                out[row:row + n, h] = a @ v
        row += n
    return out
