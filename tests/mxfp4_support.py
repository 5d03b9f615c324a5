"""Set-up of the 4-bit cache's GPU tests: pools of random codes, flattened
steps over them, and the error bound of the attention."""

from __future__ import annotations

import numpy as np
import torch

from oracle import attention as oa
from oracle import mxfp4


class Pools:
    """K and V pools of random bytes, with scales 2^lo .. 2^hi in the rows that
    `scales` was called for and noise (NaN scales among it) in the others."""

    def __init__(self, rng, num_blocks, hkv, d):
        self.hkv, self.d = hkv, d
        shape = (num_blocks, hkv * mxfp4.chunk_bytes(d))
        self.k = rng.integers(0, 256, shape, dtype=np.uint8)
        self.v = rng.integers(0, 256, shape, dtype=np.uint8)

    def scales(self, rng, slots, lo=-3, hi=2, k=True, v=True):
        for pool, is_key, wanted in ((self.k, True, k), (self.v, False, v)):
            if not wanted:
                continue
            for b in range(self.d // 32):
                place = np.array([mxfp4.scale_place(t, b, self.d, is_key) for t in range(16)])
                for h in range(self.hkv):
                    at = place[slots % 16] + h * mxfp4.chunk_bytes(self.d)
                    pool[slots // 16, at] = rng.integers(127 + lo, 128 + hi, len(slots))
        return self


class Step:
    """A flattened step of requests (query_len, past) over random pools."""

    def __init__(self, seed, reqs, heads, hkv, d, lo=-3, hi=2, spare=2, stride_pad=0,
                 table_pad=0):
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
        self.pools = Pools(rng, nb, hkv, d)
        if sum(self.seq):
            self.pools.scales(rng, np.concatenate(self.slots), lo, hi)
        self.qsl = np.concatenate([[0], np.cumsum(self.q_len)]).astype(np.int32)
        self.T = int(self.qsl[-1])
        self.q = torch.from_numpy(rng.standard_normal((self.T, heads, d + 0)).astype(np.float32)
                                  ).to(torch.bfloat16)
        self.scale = d ** -0.5
        self.stride_pad = stride_pad
        self.nan = ()   # requests whose values hold NaN: bounds per row, over its own keys

    def upload(self, device="cuda"):
        up = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(device)  # noqa: E731
        self.kc, self.vc = up(self.pools.k), up(self.pools.v)
        self.bt = up(self.table)[:, :self.width]
        self.dqsl = up(self.qsl)
        self.dseq = up(np.array(self.seq, np.int32))
        self.dpast = up(np.array(self.past, np.int32))
        wide = torch.zeros(self.T, self.H + self.stride_pad, self.d, dtype=torch.bfloat16,
                           device=device)
        self.dq = wide[:, :self.H]
        self.dq.copy_(self.q)
        return self

    def args(self):
        return (self.dq, self.kc, self.vc, self.bt, self.dqsl, self.dseq, self.dpast, self.scale)

    def history(self, r):
        k = mxfp4.read_rows(self.pools.k, self.slots[r], self.hkv, self.d, True)
        v = mxfp4.read_rows(self.pools.v, self.slots[r], self.hkv, self.d, False)
        return torch.from_numpy(k), torch.from_numpy(v)

    def reference(self):
        """(float64 output, bound on the error of a bfloat16 result) per row.

        The kernels multiply exact products in float32 (or wider), form the
        weights p = 2^(s - m) in float32 and round them to at least f16 before
        the second product.  With u = 2^-24, S = scale sum |q||k| of a row's
        worst key, A = sum_j p_j |v_j| / sum_j p_j:
          score: each of D products and a few scalings rounds at u S at most, so
            a weight is off by 2 (D + 32) u S (log2 e folded in), numerator and
            denominator both;
          weight: f16 rounds at 2^-11 (and an exponential at 2^-21) of A, or by
            2^-22 of |v_j| where p_j is below the normal f16 range (its least
            step is 2^-24; a weight may have been scaled by 2^-3 before);
          sums: 2 n u of A for n keys, at worst;
          the result: half a bfloat16 step, 2^-8 |out|; below 2^-126 a step is
            2^-133 whatever the value (8 bits down from 2^-126), half of it 2^-134.
        """
        ref = torch.zeros(self.T, self.H, self.d, dtype=torch.float64)
        tol = torch.zeros_like(ref)
        G = self.H // self.hkv
        for r in range(self.R):
            a, b = int(self.qsl[r]), int(self.qsl[r + 1])
            if a == b:
                continue
            k, v = self.history(r)
            q = self.q[a:b].double()
            # with NaN values, row by row over its own keys: 0 times NaN is NaN
            rows = [(i, i + 1) for i in range(b - a)] if r in self.nan else [(0, b - a)]
            mean = torch.zeros_like(ref[a:b])
            for i, j in rows:
                n, past = self.past[r] + j, self.past[r] + i
                ref[a + i:a + j] = oa.causal_attention_request(q[i:j], k[:n], v[:n], past, self.scale)
                mean[i:j] = oa.causal_attention_request(q[i:j], k[:n], v[:n].abs(), past, self.scale)
            n = len(k)
            seen = torch.arange(n) <= self.past[r] + torch.arange(b - a)[:, None]
            for h in range(self.H):
                s = q[:, h].abs() @ k[:, h // G].abs().T * abs(self.scale)
                s = s.masked_fill(~seen, 0).amax(1, keepdim=True)
                total = torch.stack([v[:self.past[r] + i + 1, h // G].abs().sum(0)
                                     for i in (range(b - a) if r in self.nan else [b - a - 1])])
                u = 2.0 ** -24
                tol[a:b, h] = (2.0 ** -8 * ref[a:b, h].abs()
                               + mean[:, h] * (2.0 ** -11 + 2.0 ** -20 + 4 * (self.d + 32) * u * s
                                               + 2 * n * u)
                               + 2.0 ** -22 * total + 2.0 ** -134)
        return ref, tol


def check(got, ref, tol, rows=None):
    got = got.detach().double().cpu()
    if rows is not None:
        got, ref, tol = got[rows], ref[rows], tol[rows]
    assert torch.isfinite(got).all()
    over = (got - ref).abs() - tol
    worst = over.flatten().argmax() if over.numel() else None
    assert worst is None or over.flatten()[worst] <= 0, (
        np.unravel_index(int(worst), tuple(over.shape)), float(got.flatten()[worst]),
        float(ref.flatten()[worst]), float(tol.flatten()[worst]))
