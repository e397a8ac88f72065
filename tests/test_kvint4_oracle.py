"""CPU pins of the 4-bit cache's oracle and of the arithmetic its kernels rely on."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle


def _bf16(a):
    return torch.from_numpy(np.asarray(a, dtype=np.float32)).to(torch.bfloat16)


def test_scale_is_the_smallest_bf16_that_spans_the_row():
    rng = np.random.default_rng(0)
    X = _bf16(rng.standard_normal((40, 64)) * np.exp(rng.uniform(-20, 20, (40, 1)))).double().numpy()
    codes, s, z = oracle.kv_quantize_int4_ref(X)
    for i, x in enumerate(X):
        span = Fraction(max(0.0, x.max())) - Fraction(min(0.0, x.min()))
        assert 15 * Fraction(s[i]) >= span
        below = torch.tensor([s[i]], dtype=torch.bfloat16).view(torch.int16)
        assert 15 * Fraction(float((below - 1).view(torch.bfloat16).double())) < span
    assert ((0 <= z) & (z <= 15)).all()
    back = oracle.kv_dequantize_int4_ref(codes, s, z)
    # x / s and -lo / s lie within [-15, 15] of each other, so the code is within half a step of x / s + z,
    # except where the sum of both roundings passes 15: then x was at most half a step above s (15 - z).
    assert (np.abs(back - X) <= s[:, None] / 2 * (1 + 1e-12)).all()


def test_special_rows():
    X = np.zeros((5, 64))
    X[1] = 3.0
    X[2] = -2.0
    X[3, 7] = math.inf
    X[4, 9] = math.nan
    codes, s, z = oracle.kv_quantize_int4_ref(X)
    back = oracle.kv_dequantize_int4_ref(codes, s, z)
    assert s[0] == 0 and not back[0].any()
    assert z[1] == 0 and (codes[1] == 0xFF).all()          # all codes 15
    assert z[2] == 15 or (back[2] == back[2, 0]).all()
    assert np.isnan(s[3:]).all() and np.isnan(back[3:]).all()


def test_fp32_decides_like_exact_arithmetic():
    """Quotients of two 8-bit significands: rounding the fp32 quotient to an integer never differs from rounding
    the exact one, because a quotient up to 15.5 is a half integer or at least 2^-11 away from one."""
    X = np.arange(128, 256, dtype=np.float64)
    nearest = 1.0
    for e in range(-2, 5):
        for S in range(128, 256):
            x = X * 2.0 ** e
            x = x[x <= 15.5 * S]
            if not len(x):
                continue
            frac = np.abs((x / S) % 1.0 - 0.5)     # float64: exact to 2^-48
            off = frac[(frac > 1e-12) & (x >= S / 4)]
            if len(off):
                nearest = min(nearest, off.min())
            q32 = (x.astype(np.float32) / np.float32(S)).astype(np.float32)
            exact = [round(Fraction(v) / S) for v in x]
            assert np.array_equal(np.rint(q32).astype(int), exact)
    assert nearest >= 2.0 ** -11


def test_nibbles_as_bf16_bits_are_linear():
    """A bf16 whose upper byte is zero is its low byte times 2^-133, bit 7 (the lowest exponent bit) included; scaled
    by 2^127, or by 2^123 for a nibble in bits 4..7, minus z 2^-6 it is (c - z) 2^-6 exactly in bf16."""
    bits = torch.arange(256, dtype=torch.int16)
    assert torch.equal(bits.view(torch.bfloat16).double(), bits.double() * 2.0 ** -133)
    for c in range(16):
        for z in range(16):
            v = (c - z) * 2.0 ** -6
            assert float(torch.tensor(v, dtype=torch.bfloat16)) == v
            for raw, scale in ((c, 2.0 ** 127), (16 * c, 2.0 ** 123)):
                x = float(torch.tensor([raw], dtype=torch.int16).view(torch.bfloat16).double())
                assert x * scale - z * 2.0 ** -6 == v


def test_weights_sum_to_one_a_head():
    rng = np.random.default_rng(1)
    B, Hkv, G, L, d = 2, 2, 4, 33, 64
    q, r = (rng.standard_normal((B, Hkv * G, d)) for _ in range(2))
    K, V = (rng.standard_normal((B, Hkv, L, d)) for _ in range(2))
    sl = np.array([33, 7])
    out, w = oracle.decode_weights_ref(q, r, K, V, sl, np.zeros((B, Hkv, L)))
    assert np.allclose(w.sum(-1), G) and not w[1, :, 7:].any()
    assert np.array_equal(out, oracle.decode_gqa_ref(q, r, K, V, sl))
    assert (np.abs(out) <= oracle.decode_magnitude(q, r, K, V, sl) * (1 + 1e-12)).all()


@pytest.mark.parametrize("n,budget,sinks,recent,want", [
    (4, 5, 1, 1, [0, 1, 2, 3]),
    (6, 3, 1, 1, [0, 3, 5]),
    (6, 4, 0, 0, [1, 3, 4, 5]),
    (6, 2, 1, 1, [0, 5]),
    (6, 2, 0, 0, [3, 5]),
])
def test_evict_rule(n, budget, sinks, recent, want):
    w = [0.0, 2.0, -1.0, 5.0, 2.0, 9.0]
    assert oracle.evict_ref(w, n, budget, sinks, recent).tolist() == want


def test_evict_ties_and_nan():
    w = [1.0, math.nan, 1.0, -math.inf, 1.0, -0.0, 0.0]
    assert oracle.evict_ref(w, 7, 2, 0, 0).tolist() == [0, 2]
    assert oracle.evict_ref(w, 7, 4, 0, 0).tolist() == [0, 2, 4, 5]
    assert oracle.evict_ref(w, 7, 6, 0, 0).tolist() == [0, 2, 3, 4, 5, 6]
