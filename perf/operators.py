"""Cases, plain forms and 64-bit values of the operators of the 4-bit paged cache.

The operators: the step's tables on the device (`build_step_metadata`), the
quantising cache write (`reshape_and_cache_mxfp4`), its read-back
(`gather_cache_mxfp4`) and attention over the 4-bit cache
(`paged_attention_varlen_mxfp4`: rows of one new token, and prefill chunks).

A cache is uint8 [num_blocks, Hkv * 17 D / 2].  One block holds 16 tokens; KV
head h owns bytes [h * 17 D / 2, (h + 1) * 17 D / 2): 16 rows of D / 2 bytes of
e2m1 codes (even position in the low nibble), then 16 * D / 32 bytes of e8m0
scales, one per 32 dimensions of a row.  With b = d // 32:
  key code of dim d:    byte ((d % 32) // 8) * D / 8 + 4 b + (d % 8) // 2 of its row
  value code of dim d:  byte ((d % 32) // 4) * D / 16 + 2 b + (d % 4) // 2 of its row
  key scale (t, b):     t * D / 32 + b
  value scale (t, b):   (t // 2) * D / 16 + (b // 2) * 4 + (t % 2) * 2 + b % 2
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
        # one decoding request gets one more token: the smallest call, all latency
        dict(name="tables_one_token", op="tables", reqs=1, new_lo=1, new_hi=1, held_hi=4096, width=2048),
        # a step that admits a thousand short prompts and decodes the rest: 16-token-budget
        # arithmetic for some 130000 tokens
        dict(name="tables_prompts", op="tables", reqs=1024, new_lo=1, new_hi=256, held_hi=4096, width=512),
        # the new tokens of a 64-request decode step, Llama-3-8B KV heads
        dict(name="write_decode64", op="write", tokens=64, hkv=8, d=128, dtype="bf16", fused=True, pad=0),
        # the largest prefill step of the serving trace (8192-token budget), K and V inside a
        # fused QKV projection's rows
        dict(name="write_8192", op="write", tokens=8192, hkv=8, d=128, dtype="bf16", fused=True, pad=0),
        # float32 rows, odd counts, padding tokens
        dict(name="write_f32_odd", op="write", tokens=1337, hkv=5, d=64, dtype="f32", fused=False, pad=9),
        # a request's history leaves the 4-bit pool (16384 tokens, as bf16)
        dict(name="read_16384", op="read", tokens=16384, hkv=8, d=128, dtype="bf16", pad=0),
        # an odd number of small float32 rows
        dict(name="read_f32_odd", op="read", tokens=777, hkv=2, d=64, dtype="f32", pad=5),
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
    op = rng.choice(["tables", "write", "read", "decode", "decode", "prefill", "mixed"])
    if op == "tables":
        reqs = _log(rng, 1, 4096)
        new_hi = _log(rng, 1, max(1, min(16384, 131072 // reqs)))
        return dict(op="tables", reqs=reqs, new_lo=rng.choice([0, 1, 1]), new_hi=new_hi,
                    held_hi=_log(rng, 1, 16384 if reqs <= 1024 else 4096), width=2048 if reqs <= 1024 else 512)
    if op in ("write", "read"):
        d = rng.choice([64, 128])
        case = dict(op=op, tokens=_log(rng, 1, 16384 if op == "read" else 8192), hkv=rng.choice([1, 2, 3, 4, 5, 8]), d=d,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), pad=rng.choice([0, 0, 1, 7]))
        if op == "write":
            case["fused"] = rng.choice([True, False])
        if case["dtype"] == "f32":
            case["tokens"] = max(1, case["tokens"] // 2)
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
    """The case's own request lengths (host integers, the same for every seed)."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    if case["op"] == "tables":
        held = [rng.randint(0, case["held_hi"]) for _ in range(case["reqs"])]
        new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["reqs"])]
        new[0] = max(1, new[0])
        return held, new
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
    if op == "tables":
        held, new = _lengths(case)
        need = sum(_blocks(h + s) - _blocks(h) for h, s in zip(held, new))
        return {"bytes": 16 * sum(new) + 8 * need + 16 * len(held) + 32, "flops": 0}
    if op in ("write", "read"):
        values = 2 * case["tokens"] * case["hkv"] * case["d"]
        wide = values * (4 if case["dtype"] == "f32" else 2)
        small = values * 17 // 32
        # a write is followed by its read-back: rows in, rows out, the cache written and read
        return {"bytes": (2 * wide + 2 * small if op == "write" else wide + small) + 8 * case["tokens"], "flops": 0}
    q, past = _lengths(case)
    ctx = sum(p + n for p, n in zip(past, q) if n)
    rows = sum(q)
    pairs = sum(n * p + n * (n + 1) // 2 for p, n in zip(past, q))
    cache = ctx * 2 * case["hkv"] * case["d"] * 17 // 32
    return {"bytes": cache + 2 * rows * case["heads"] * case["d"] * 2 + 4 * _blocks(ctx),
            "flops": 4 * pairs * case["heads"] * case["d"]}


# ------------------------------------------------- the cache, in torch operations
def _chunk(d):
    return 17 * d // 2


def _power(e):
    """2^(e - 127) as float32, from its bits (e in [0, 254])."""
    return torch.where(e == 0, 1 << 22, e.int() << 23).int().view(torch.float32)


def _quantise(x):
    """float32 [..., D] -> (codes uint8 [..., D], scale bytes uint8 [..., D / 32])."""
    b = x.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    finite = torch.isfinite(b).all(-1)
    # floor(log2 amax) is the exponent field of a normal float32
    expo = (torch.where(finite, amax, 1.0).contiguous().view(torch.int32) >> 23) - 127
    e = torch.where(amax > 0, (expo - 2 + 127).clamp(1, 254), 127)
    y = (b * _power(254 - e).unsqueeze(-1)).abs()
    # round to nearest on {0, .5, 1, 1.5, 2, 3, 4, 6}, ties to the even code
    code = ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5))
    code = code + 8 * torch.signbit(b).to(torch.uint8)
    code = torch.where(finite.unsqueeze(-1), code, 0)
    return code.flatten(-2), torch.where(finite, e, 255).to(torch.uint8)


def _write(pool, codes, scales, slots, d, is_key):
    """Rows codes [n, Hkv, D] / scales [n, Hkv, D / 32] to their slots of a pool."""
    hkv, nb = codes.shape[1], d // 32
    p = pool.view(pool.shape[0], hkv, _chunk(d))
    c = codes.unflatten(-1, (nb, 4, 8)) if is_key else codes.unflatten(-1, (nb, 8, 4))
    c = c.transpose(-3, -2).flatten(-3)
    blk, off = slots // BS, slots % BS
    p[:, :, :BS * d // 2].unflatten(-1, (BS, d // 2))[blk, :, off] = c[..., 0::2] | (c[..., 1::2] << 4)
    s = p[:, :, BS * d // 2:]
    if is_key:
        s.unflatten(-1, (BS, nb))[blk, :, off] = scales
    else:
        s.unflatten(-1, (BS // 2, nb // 2, 2, 2))[blk, :, off // 2, :, off % 2] = scales.unflatten(-1, (-1, 2))


_TABLE = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _read(blocks, hkv, d, is_key):
    """uint8 [..., block bytes] -> float32 [..., 16 tokens, Hkv, D]."""
    nb = d // 32
    p = blocks.unflatten(-1, (hkv, _chunk(d)))
    raw, s = p[..., :BS * d // 2], p[..., BS * d // 2:]
    c = torch.stack((raw & 15, raw >> 4), -1).flatten(-2)
    c = c.unflatten(-1, (BS, 4, nb, 8)) if is_key else c.unflatten(-1, (BS, 8, nb, 4))
    c = c.transpose(-3, -2).flatten(-2)                                 # [..., Hkv, 16, nb, 32]
    x = torch.tensor(_TABLE, device=blocks.device)[c.int()]
    s = s.unflatten(-1, (BS, nb)) if is_key else \
        s.unflatten(-1, (BS // 2, nb // 2, 2, 2)).transpose(-3, -2).flatten(-2).flatten(-3, -2)
    x *= torch.where(s == 255, torch.nan, _power(s)).unsqueeze(-1)
    return x.flatten(-2).transpose(-3, -2)


# --------------------------------------------------------------------- inputs
def _values(gen, tokens, hkv, d):
    """Rows as a K or V projection gives them: a scale per channel (a few loud
    ones), a scale per token."""
    g = dict(generator=gen, device=DEV)
    channel = torch.exp2(torch.randn(hkv, d, **g)) * torch.where(torch.rand(hkv, d, **g) < 0.02, 8.0, 0.5)
    x = torch.randn(tokens, hkv, d, **g)
    return x * channel * torch.exp2(0.5 * torch.randn(tokens, 1, 1, **g))


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed * 7919 + 17)
    g = dict(generator=gen, device=DEV)
    op = case["op"]
    if op == "tables":
        held, new = _lengths(case)
        need = sum(_blocks(h + s) - _blocks(h) for h, s in zip(held, new))
        have = [_blocks(h) for h in held]
        pool = sum(have) + need + 64
        ids = torch.randperm(pool, **g).to(torch.int32)
        width = max(case["width"], max(_blocks(h + s) for h, s in zip(held, new)))
        table = torch.full((len(held), width), -1, dtype=torch.int32, device=DEV)
        col = torch.arange(width, device=DEV)
        mask = col < torch.tensor(have, device=DEV).unsqueeze(1)
        table[mask] = ids[:sum(have)]
        free = ids[sum(have):]
        # the ring of free blocks, some way round: head and tail only ever grow
        head = int(torch.randint(0, 1 << 20, (1,), generator=gen, device=DEV))
        ring = torch.empty_like(free)
        ring[(head + torch.arange(len(free), device=DEV)) % len(free)] = free
        i32 = dict(dtype=torch.int32, device=DEV)
        tokens = sum(new)
        return dict(case=case, new=torch.tensor(new, **i32), held=torch.tensor(held, **i32), table=table, ring=ring,
                    state=torch.tensor([head, head + len(free), 0, 0], dtype=torch.int64, device=DEV),
                    state_out=torch.zeros(4, dtype=torch.int64, device=DEV), tokens=tokens + (-tokens) % 8,
                    qsl=torch.empty(len(new) + 1, **i32), seq=torch.empty(len(new), **i32),
                    slots=torch.empty(tokens + (-tokens) % 8, dtype=torch.int64, device=DEV),
                    positions=torch.empty(tokens + (-tokens) % 8, dtype=torch.int64, device=DEV))
    hkv, d = case["hkv"], case["d"]
    size = hkv * _chunk(d)
    if op in ("write", "read"):
        t, dt = case["tokens"], _dtype(case)
        nblk = _blocks(t) + 8
        kpool = torch.randint(0, 256, (nblk, size), dtype=torch.uint8, **g)
        vpool = torch.randint(0, 256, (nblk, size), dtype=torch.uint8, **g)
        slots = torch.randperm(nblk * BS, **g)[:t].contiguous()
        if case["pad"]:
            slots[torch.randperm(t, **g)[:case["pad"]]] = -1
        s = dict(case=case, kpool=kpool, vpool=vpool, slots=slots,
                 kout=torch.zeros(t, hkv, d, dtype=dt, device=DEV), vout=torch.zeros(t, hkv, d, dtype=dt, device=DEV))
        k, v = _values(gen, t, hkv, d).to(dt), _values(gen, t, hkv, d).to(dt)
        if op == "write":
            if case["fused"]:   # [q heads | k heads | v heads] rows of one projection
                rows = torch.zeros(t, 6 * hkv, d, dtype=dt, device=DEV)
                rows[:, 4 * hkv:5 * hkv], rows[:, 5 * hkv:] = k, v
                k, v = rows[:, 4 * hkv:5 * hkv], rows[:, 5 * hkv:]
            s.update(k=k, v=v)
        else:
            live = slots >= 0
            _write(kpool, *(x[live] for x in _quantise(k.float())), slots[live], d, True)
            _write(vpool, *(x[live] for x in _quantise(v.float())), slots[live], d, False)
        return s
    q, past = _lengths(case)
    seq = [p + n for p, n in zip(past, q)]
    count = [_blocks(n) for n in seq]
    used = sum(count)
    nblk = used + used // 4 + 4
    # blocks scattered over the pool; what no token has written is left as it was: noise
    kpool = torch.randint(0, 256, (nblk, size), dtype=torch.uint8, **g)
    vpool = torch.randint(0, 256, (nblk, size), dtype=torch.uint8, **g)
    width = max(count + [1])
    table = torch.full((len(q), width), -1, dtype=torch.int32, device=DEV)
    col = torch.arange(width, device=DEV)
    table[col < torch.tensor(count, device=DEV).unsqueeze(1)] = torch.randperm(nblk, **g)[:used].to(torch.int32)
    lens = torch.tensor(seq, device=DEV)
    first = torch.cumsum(lens, 0) - lens
    total = sum(seq)
    for lo in range(0, total, 1 << 17):
        i = torch.arange(lo, min(total, lo + (1 << 17)), device=DEV)
        r = torch.searchsorted(torch.cumsum(lens, 0), i, right=True)
        p = i - first[r]
        slots = table[r, p // BS].long() * BS + p % BS
        _write(kpool, *_quantise(_values(gen, len(i), hkv, d)), slots, d, True)
        _write(vpool, *_quantise(_values(gen, len(i), hkv, d)), slots, d, False)
    i32 = dict(dtype=torch.int32, device=DEV)
    rows = sum(q)
    return dict(case=case, kpool=kpool, vpool=vpool, table=table,
                q=torch.randn(rows, case["heads"], d, **g).to(torch.bfloat16),
                out=torch.empty(rows, case["heads"], d, dtype=torch.bfloat16, device=DEV),
                qsl=torch.tensor(np.concatenate([[0], np.cumsum(q)]), **i32),
                seq=torch.tensor(seq, **i32), past=torch.tensor(past, **i32), longest=max(q), scale=d ** -0.5)


# ------------------------------------------------------------------ plain forms
def _plain_tables(s):
    new, held, table, ring = s["new"].long(), s["held"].long(), s["table"], s["ring"]
    head, tail = s["state"][0], s["state"][1]
    width, cap = table.shape[1], ring.shape[0]
    have = (held + BS - 1) // BS
    need = (held + new + BS - 1) // BS - have
    first = torch.cumsum(need, 0) - need
    total = need.sum()
    ok = (total <= tail - head) & (have + need <= width).all()
    col = torch.arange(width, device=table.device)
    mine = (col >= have[:, None]) & (col < (have + need)[:, None]) & ok
    at = torch.where(mine, (head + first[:, None] + col - have[:, None]) % cap, 0)
    table.copy_(torch.where(mine, ring[at], table))
    new = torch.where(ok, new, 0)
    ends = torch.cumsum(new, 0)
    qsl = torch.cat((torch.zeros(1, dtype=torch.int64, device=table.device), ends))
    t = torch.arange(s["tokens"], device=table.device)
    r = torch.searchsorted(ends, t, right=True)
    live = r < len(ends)
    r = r.clamp(max=len(ends) - 1)
    pos = torch.where(live, held[r] + t - qsl[r], 0)
    slot = torch.where(live, table[r, pos // BS].long() * BS + pos % BS, -1)
    after = torch.stack((head + torch.where(ok, total, 0), tail))
    return [table, qsl.int(), (held + new).int(), slot, pos, after]


def _rows_of(pool, slots, hkv, d, is_key, dt):
    at = slots.clamp(min=0)
    x = _read(pool[at // BS], hkv, d, is_key)
    x = x[torch.arange(len(at), device=at.device), at % BS]
    return torch.where((slots >= 0)[:, None, None], x, 0).to(dt)


def _plain_write(s):
    d, live = s["case"]["d"], s["slots"] >= 0
    _write(s["kpool"], *(x[live] for x in _quantise(s["k"].float())), s["slots"][live], d, True)
    _write(s["vpool"], *(x[live] for x in _quantise(s["v"].float())), s["slots"][live], d, False)


def _plain_read(s):
    c = s["case"]
    return [_rows_of(s["kpool"], s["slots"], c["hkv"], c["d"], True, _dtype(c)),
            _rows_of(s["vpool"], s["slots"], c["hkv"], c["d"], False, _dtype(c))]


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
    k = _read(s["kpool"][s["table"][lo:hi].clamp(min=0).long()], c["hkv"], c["d"], True).flatten(1, 2).transpose(1, 2)
    v = _read(s["vpool"][s["table"][lo:hi].clamp(min=0).long()], c["hkv"], c["d"], False).flatten(1, 2).transpose(1, 2)
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
    op = s["case"]["op"]
    if own:
        import paged_kv_cache_36_gb300 as pkv
        if op == "tables":
            pkv.build_step_metadata(s["new"], s["held"], s["table"], s["ring"], s["state"], s["tokens"],
                                    free_state_out=s["state_out"], query_start_loc=s["qsl"], seq_lens=s["seq"],
                                    slot_mapping=s["slots"], positions=s["positions"])
            return [s["table"], s["qsl"], s["seq"], s["slots"], s["positions"], s["state_out"][:2]]
        if op in ("write", "read"):
            if op == "write":
                pkv.reshape_and_cache_mxfp4(s["k"], s["v"], s["kpool"], s["vpool"], s["slots"])
            pkv.gather_cache_mxfp4(s["kpool"], s["vpool"], s["slots"], s["kout"], s["vout"])
            return [s["kout"], s["vout"]]
        if "workspace" not in s:   # kept from call to call, as a server keeps it
            s["workspace"] = pkv.new_workspace_mxfp4(s["case"]["heads"], s["case"]["hkv"], s["case"]["d"])
        return pkv.paged_attention_varlen_mxfp4(s["q"], s["kpool"], s["vpool"], s["table"], s["qsl"], s["seq"],
                                                s["past"], s["scale"], out=s["out"], workspace=s["workspace"],
                                                max_query_len=s["longest"])
    if op == "tables":
        return _plain_tables(s)
    if op in ("write", "read"):
        if op == "write":
            _plain_write(s)
        return _plain_read(s)
    _plain_rows(s, 0, s["case"]["prompts"])
    _plain_rows(s, s["case"]["prompts"], s["case"]["prompts"] + s["case"]["decodes"])
    return s["out"]


# ------------------------------------------------------------- 64-bit definition
def _grid64(x):
    """The values that 4-bit rows of x (float64 [..., D]) stand for, by search on the grid."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    _, ex = torch.frexp(amax)                                  # amax = m 2^ex, m in [1/2, 1)
    k = (ex - 1 - 2).clamp(-126, 127)
    k = torch.where(amax > 0, k, 0)
    unit = ((k.long() + 1023) << 52).view(torch.float64)       # 2^k
    y = (b / unit).abs()
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    # nearest; of two equally near, the one of even index
    best, near = torch.zeros_like(y), torch.full_like(y, torch.inf)
    for i in (0, 2, 4, 6, 1, 3, 5, 7):
        dist = (y - grid[i]).abs()
        closer = dist < near
        best, near = torch.where(closer, grid[i], best), torch.where(closer, dist, near)
    return (torch.copysign(best, b) * unit).reshape(x.shape)


def _values64(pool, slots, hkv, d, is_key):
    """float64 [n, Hkv, D] of the given slots, byte by byte from the layout."""
    dim = torch.arange(d, device=DEV)
    b = dim // 32
    t = slots % BS
    if is_key:
        byte, half = (dim % 32) // 8 * (d // 8) + 4 * b + (dim % 8) // 2, dim % 2
        scale = t[:, None] * (d // 32) + b
    else:
        byte, half = (dim % 32) // 4 * (d // 16) + 2 * b + (dim % 4) // 2, dim % 2
        scale = (t // 2 * (d // 16))[:, None] + b // 2 * 4 + (t % 2 * 2)[:, None] + b % 2
    head = torch.arange(hkv, device=DEV) * _chunk(d)
    blk = (slots // BS)[:, None, None]
    code = pool[blk, head[:, None] + (t[:, None] * (d // 2) + byte)[:, None, :]]
    code = torch.where(half == 0, code % 16, code // 16).int()
    mag, man = code % 8 // 2, code % 2
    x = torch.where(mag == 0, man * 0.5, (1 + man * 0.5) * torch.exp2((mag - 1).double()))
    x = torch.where(code >= 8, -x, x)
    return x * torch.exp2(pool[blk, head[:, None] + (BS * d // 2 + scale)[:, None, :]].double() - 127)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "tables":
        held, new = _lengths(case)
        table, ring, slots, pos = s["table"].cpu().numpy(), s["ring"].cpu().numpy(), [], []
        head, tail = (int(x) for x in s["state"][:2])
        for r, (h, n) in enumerate(zip(held, new)):
            for p in range(h, h + n):
                if p % BS == 0:
                    table[r, p // BS] = ring[head % len(ring)]
                    head += 1
                slots.append(int(table[r, p // BS]) * BS + p % BS)
                pos.append(p)
        fill = s["tokens"] - len(slots)
        return [table, np.concatenate([[0], np.cumsum(new)]).astype(np.int32), np.array(held, np.int32) + np.array(new, np.int32),
                np.array(slots + [-1] * fill), np.array(pos + [0] * fill), np.array([head, tail])]
    hkv, d = case["hkv"], case["d"]
    if op in ("write", "read"):
        live = (s["slots"] >= 0)[:, None, None]
        if op == "write":
            got = [_grid64(s["k"].double()), _grid64(s["v"].double())]
        else:
            at = s["slots"].clamp(min=0)
            got = [_values64(s["kpool"], at, hkv, d, True), _values64(s["vpool"], at, hkv, d, False)]
        return [torch.where(live, x, 0.0) for x in got]
    q_len, past = _lengths(case)
    group = case["heads"] // hkv
    out = torch.zeros(sum(q_len), case["heads"], d, dtype=torch.float64, device=DEV)
    row = 0
    for r, (n, p) in enumerate(zip(q_len, past)):
        if n == 0:
            continue
        j = torch.arange(p + n, device=DEV)
        slots = s["table"][r, j // BS].long() * BS + j % BS
        k, v = _values64(s["kpool"], slots, hkv, d, True), _values64(s["vpool"], slots, hkv, d, False)
        hide = j[None, :] > p + torch.arange(n, device=DEV)[:, None]
        for h in range(case["heads"]):
            a = s["q"][row:row + n, h].double() @ k[:, h // group].T * s["scale"]
            a = torch.softmax(a.masked_fill(hide, -torch.inf), -1)
            out[row:row + n, h] = a @ v[:, h // group]
        row += n
    return out
