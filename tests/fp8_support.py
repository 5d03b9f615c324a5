"""Set-up of the 8-bit cache's GPU tests: pools of random codes, flattened steps over
them, and the error bound of the attention."""

from __future__ import annotations

import numpy as np
import torch

from oracle import fp8


def codes_of(x, e):
    """e4m3 codes of float64 numbers at scale bytes e: oracle.fp8.code of whole arrays."""
    grid = fp8.TABLE[:fp8.NAN]
    y = np.abs(np.where(np.isfinite(x), x, 0.0)) * np.exp2(127.0 - e)
    mids = (grid[1:] + grid[:-1]) / 2
    i = np.searchsorted(mids, y)        # mids[i - 1] < y <= mids[i]
    tie = (i < len(mids)) & (y == mids[np.minimum(i, len(mids) - 1)])
    i += tie & (i % 2 == 1)
    return np.where(np.isfinite(x), i + 128 * np.signbit(x), fp8.NAN).astype(np.uint8)


def write_many(pool, slots, rows, is_key):
    """oracle.fp8.write, block by block at once."""
    _, hkv, d = rows.shape
    slots = np.asarray(slots)
    at = np.array([[fp8.place(t, i, d, is_key) for i in range(d)] for t in range(16)])
    live, first = np.unique(slots[::-1], return_index=True)     # (the last of equal ones)
    token = len(slots) - 1 - first
    token, live = token[live >= 0], live[live >= 0]
    blocks, of = np.unique(live // 16, return_inverse=True)
    x = rows[token]
    amax = np.zeros((len(blocks), hkv))
    np.maximum.at(amax, of, np.abs(np.where(np.isfinite(x), x, 0.0)).max(-1))
    m, ex = np.frexp(amax)
    e = np.where(amax > 0, np.clip(127 + ex - 9 + (m > 0.875), fp8.LOW, fp8.HIGH), fp8.LOW)
    chunks = pool.reshape(len(pool), hkv, -1)[blocks]
    old = np.clip(chunks[..., 16 * d].astype(int), fp8.LOW, fp8.HIGH)
    anew = np.zeros(len(blocks), bool)
    anew[of[live % 16 == 0]] = True
    e = np.where(anew[:, None], e, np.maximum(e, old))
    codes = chunks[..., at]                                     # [blocks, hkv, 16, d]
    down = codes_of(fp8.TABLE[codes & 127] * np.exp2(np.minimum(old - e, 0).astype(float))[..., None, None],
                    np.full(codes.shape, 127))
    down = np.where(down == fp8.NAN, fp8.NAN, down | codes & 128)
    codes = np.where((e > old)[..., None, None], down, codes)
    codes[anew] = 0
    codes[of[:, None], np.arange(hkv), (live % 16)[:, None]] = codes_of(x, e[of][..., None])
    chunks[..., at] = codes
    chunks[..., 16 * d:] = 0
    chunks[..., 16 * d] = e
    pool.reshape(len(pool), hkv, -1)[blocks] = chunks


class Step:
    """A flattened step of requests (query_len, past) over pools of random codes: those of the
    requests' tokens are numbers with scales 2^lo .. 2^hi, everything else is noise (NaN
    codes and any scale among it)."""

    def __init__(self, seed, reqs, heads, hkv, d, lo=-9, hi=-5, spare=2, stride_pad=0, table_pad=0):
        rng = self.rng = np.random.default_rng(seed)
        self.q_len = [n for n, _ in reqs]
        self.past = [p for _, p in reqs]
        self.seq = [n + p for n, p in reqs]
        self.R, self.H, self.hkv, self.d = len(reqs), heads, hkv, d
        counts = [-(-s // 16) for s in self.seq]
        nb = sum(counts) + spare
        ids = rng.permutation(nb).astype(np.int32)
        self.width = max(counts + [1])
        self.table = np.full((self.R, self.width + table_pad), -1, np.int32)
        self.slots = []
        at = 0
        for r, c in enumerate(counts):
            self.table[r, :c] = ids[at:at + c]
            at += c
            p = np.arange(self.seq[r])
            self.slots.append(self.table[r, p // 16].astype(np.int64) * 16 + p % 16)
        self.k, self.v = (rng.integers(0, 256, (nb, hkv * fp8.chunk_bytes(d)), dtype=np.uint8) for _ in "kv")
        self.at = {key: np.array([[fp8.place(t, i, d, key) for i in range(d)] for t in range(16)])
                   for key in (True, False)}
        live = np.concatenate(self.slots) if self.slots else np.zeros(0, np.int64)
        for pool, key in ((self.k, True), (self.v, False)):
            for h in range(hkv):
                base = h * fp8.chunk_bytes(d)
                codes = rng.integers(0, 254, (len(live), d), dtype=np.uint8)
                pool[(live // 16)[:, None], base + self.at[key][live % 16]] = codes + (codes >= 127)
                blocks = np.unique(live // 16)
                pool[blocks, base + 16 * d] = rng.integers(127 + lo, 128 + hi, len(blocks))
        self.qsl = np.concatenate([[0], np.cumsum(self.q_len)]).astype(np.int32)
        self.T = int(self.qsl[-1])
        self.q = torch.from_numpy(rng.standard_normal((self.T, heads, d)).astype(np.float32)).to(torch.bfloat16)
        self.scale = d ** -0.5
        self.stride_pad = stride_pad

    def set(self, pool, key, r, pos, h, dim, code):
        """Codes of request r's tokens at pos (integers or an array)."""
        s = self.slots[r][pos]
        pool[s // 16, h * fp8.chunk_bytes(self.d) + self.at[key][s % 16, dim]] = code

    def set_scale(self, pool, r, block, h, e):
        pool[self.table[r, block], h * fp8.chunk_bytes(self.d) + 16 * self.d] = e

    def upload(self, device="cuda"):
        up = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(device)  # noqa: E731
        self.kc, self.vc = up(self.k), up(self.v)
        self.bt = up(self.table)[:, :self.width]
        self.dqsl = up(self.qsl)
        self.dseq = up(np.array(self.seq, np.int32))
        self.dpast = up(np.array(self.past, np.int32))
        wide = torch.zeros(self.T, self.H + self.stride_pad, self.d, dtype=torch.bfloat16, device=device)
        self.dq = wide[:, :self.H]
        self.dq.copy_(self.q)
        return self

    def args(self):
        return (self.dq, self.kc, self.vc, self.bt, self.dqsl, self.dseq, self.dpast, self.scale)

    def history(self, r):
        return tuple(torch.from_numpy(fp8.read_rows(pool, self.slots[r], self.hkv, self.d, key))
                     for pool, key in ((self.k, True), (self.v, False)))

    def reference(self):
        """(float64 output, bound on the error of a bfloat16 result) per row; NaN where a
        key or value that the row sees is NaN.

        K, V and q are exact in bfloat16, so products are exact and sums float32.  With u =
        2^-24, S = scale sum |q||k| of a row's worst key and A = sum_j p_j |v_j| / sum_j p_j:
          score: each of D products and a few scalings rounds at u S at most, so a weight is
            off by 2 (D + 32) u S (log2 e folded in), numerator and denominator both;
          weight: half a bfloat16 step, 2^-8 of A in the numerator, and (the denominator sums the
            rounded weights) 2^-8 |out|: sum_j p_j d_j (v_j - out) with |d_j| <= 2^-8 is at most
            2^-8 (A + |out|).  (And an exponential's 2^-21.)  Weights are formed as 2^(s - m) with m at most 24 above the row's largest score, and vanish below
            2^-126 (the exponential flushes there): where p_j is below 2^-102 of the largest
            nothing is left of it, 2^-102 |v_j|;
          sums: 2 n u of A for n keys, at worst;
          the result: half a bfloat16 step, 2^-8 |out|; below 2^-126 half of 2^-133.
        """
        ref = torch.zeros(self.T, self.H, self.d, dtype=torch.float64)
        tol = torch.zeros_like(ref)
        G, u = self.H // self.hkv, 2.0 ** -24
        for r in range(self.R):
            a, b = int(self.qsl[r]), int(self.qsl[r + 1])
            if a == b:
                continue
            k, v = self.history(r)
            q = self.q[a:b].double()
            n = len(k)
            seen = torch.arange(n) <= self.past[r] + torch.arange(b - a)[:, None]
            for h in range(self.H):
                kh, vh = k[:, h // G], v[:, h // G]
                s = (q[:, h] @ kh.T * self.scale).masked_fill(~seen, -torch.inf)
                p = torch.softmax(s, -1)
                nan = (seen.double() @ vh.isnan().double()) > 0     # by row and dimension
                vh = vh.nan_to_num(0.0)
                out = p @ vh
                worst = (q[:, h].abs() @ kh.abs().T * abs(self.scale)).masked_fill(~seen, 0).amax(1, keepdim=True)
                mean = p @ vh.abs()
                ref[a:b, h] = out.masked_fill(nan, torch.nan)
                tol[a:b, h] = (2.0 ** -7 * out.abs()
                               + mean * (2.0 ** -8 + 2.0 ** -20 + 4 * (self.d + 32) * u * worst + 2 * n * u)
                               + 2.0 ** -102 * (seen.double() @ vh.abs()) + 2.0 ** -134)
        return ref, tol


def check(got, ref, tol, rows=None):
    got = got.detach().double().cpu()
    if rows is not None:
        got, ref, tol = got[rows], ref[rows], tol[rows]
    nan = ref.isnan()
    assert torch.equal(got.isnan(), nan), (got.isnan().sum(), nan.sum())
    over = ((got - ref).abs() - tol).masked_fill(nan, -1.0)
    worst = over.flatten().argmax() if over.numel() else None
    assert worst is None or over.flatten()[worst] <= 0, (
        np.unravel_index(int(worst), tuple(over.shape)), float(got.flatten()[worst]),
        float(ref.flatten()[worst]), float(tol.flatten()[worst]))
