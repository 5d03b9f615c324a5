"""The table of rotary angles against float64: an entry is the float32 nearest to its value,
but for the errors of the float32 sine and cosine (2^-23 of the factor in all)."""

import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import fp8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n, rd, start, base, scaling, factor, length, low, high, attention", [
    (1, 2, 0, 1e4, "none", 1.0, 0, 1.0, 32.0, None), (513, 128, 0, 1e4, "none", 1.0, 0, 1.0, 32.0, None),
    (33, 64, 1000000, 5e5, "none", 1.0, 0, 1.0, 32.0, 0.5), (100, 96, 3, 1e4, "linear", 4.0, 0, 1.0, 32.0, None),
    (77, 64, 131000, 1e4, "ntk", 8.0, 0, 1.0, 32.0, None), (50, 4, 9, 1e4, "ntk", 2.5, 0, 1.0, 32.0, None),
    (300, 128, 100000, 5e5, "parts", 8.0, 8192, 1.0, 4.0, None), (64, 512, 7, 1e4, "parts", 3.0, 300, 0.5, 32.0, None),
    (200, 64, 50000, 1e4, "yarn", 16.0, 4096, 1.0, 32.0, None), (20, 8, 0, 1e4, "yarn", 1.0, 5, 1.0, 4.0, 2.0),
    (5, 6, (1 << 26) - 5, 1e6, "yarn", 64.0, 32768, 1.0, 32.0, None)])
def test_table(n, rd, start, base, scaling, factor, length, low, high, attention):
    import paged_kv_cache_36_gb300 as pkv
    got = pkv.build_cos_sin_cache(n, rd, base=base, scaling=scaling, factor=factor, original_max_position=length,
                                  low=low, high=high, attention_factor=attention, start=start)
    if attention is None:
        attention = 0.1 * np.log(factor) + 1.0 if scaling == "yarn" else 1.0
    want = fp8.cos_sin(n, rd, base, scaling, factor, length, low, high, attention, start)
    assert got.shape == (n, rd) and got.dtype is torch.float32
    # 2^-23 of the factor (documented), and what a 64-bit angle of 2^26 is off by itself
    assert np.abs(got.double().cpu().numpy() - want).max() <= attention * (2.0 ** -23 + (start + n) * 2.0 ** -51)


TAU = Fraction("6.28318530717958647692528676655900576839433879875021164194989")


def _exact(n, rd, start, freqs, attention):
    """float64 [n, rd] from angles in turns, 64 bits behind the point (of 2^26 positions 2^-39)."""
    turns = np.array([round(Fraction(f) / TAU * 2 ** 64) % 2 ** 64 for f in freqs], np.uint64)
    with np.errstate(over="ignore"):
        rest = (np.arange(start, start + n, dtype=np.uint64)[:, None] * turns).view(np.int64)
    angle = rest.astype(np.float64) * (2.0 ** -64 * 2 * math.pi)
    return attention * np.concatenate([np.cos(angle), np.sin(angle)], 1)


@pytest.mark.parametrize("scaling, factor, attention, start", [
    ("yarn", 8.0, None, 0), ("yarn", 32.0, None, 100000), ("yarn", 40.0, None, 0), ("linear", 4.0, 0.7, 1 << 20),
    ("none", 1.0, 1.069, 0), ("parts", 8.0, -1.45, (1 << 26) - 40000), ("none", 1.0, 1.0, 3), ("ntk", 4.0, 1e-30, 0),
    ("none", 1.0, 3.4e38, 0)])
def test_the_documented_bound(scaling, factor, attention, start):
    """2^-23 of the factor, over 5 million entries."""
    import paged_kv_cache_36_gb300 as pkv
    n, rd = 40000, 128
    got = pkv.build_cos_sin_cache(n, rd, scaling=scaling, factor=factor, original_max_position=4096,
                                  attention_factor=attention, start=start)
    if attention is None:
        attention = 0.1 * np.log(factor) + 1.0
    want = _exact(n, rd, start, fp8.frequencies(rd, 1e4, scaling, factor, 4096, 1.0, 32.0), attention)
    assert np.abs(got.double().cpu().numpy() - want).max() <= abs(attention) * 2.0 ** -23


def test_extending_and_rotating_with_it():
    """A table made in two parts is the table made at once, and RoPE reads it."""
    import paged_kv_cache_36_gb300 as pkv
    whole = pkv.build_cos_sin_cache(300, 64, scaling="linear", factor=2.0)
    parts = torch.empty_like(whole)
    s = torch.cuda.Stream()
    pkv.build_cos_sin_cache(200, 64, scaling="linear", factor=2.0, out=parts[:200], stream=s)
    pkv.build_cos_sin_cache(100, 64, scaling="linear", factor=2.0, start=200, out=parts[200:], stream=s)
    s.synchronize()
    assert torch.equal(whole, parts)
    q = torch.randn(3, 2, 64, device="cuda")
    k = torch.randn(3, 1, 64, device="cuda")
    want = q.clone()
    kc = torch.zeros(1, 16, 1, 64, device="cuda")
    pos, slots = torch.tensor([0, 299, 7], device="cuda"), torch.tensor([0, 1, 2], device="cuda")
    pkv.rope_reshape_and_cache(pos, want, k, k, kc, kc.clone(), slots, whole)
    out = torch.empty_like(q)
    k8, v8 = pkv.new_cache_fp8(1, 1, 64)
    pkv.rope_reshape_and_cache_fp8(pos, q, k, k, k8, v8, slots, parts, query_out=out)
    assert ((out - want).abs() <= 2.0 ** -22 * q.abs().amax()).all()
