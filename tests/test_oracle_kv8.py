"""The 8-bit cache's oracle against torch's own conversions, exact rationals and brute force."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import bf16, kv8


def test_e4m3_rounding_is_torchs():
    y = np.concatenate([np.linspace(-448, 448, 200001), kv8._E4M3, -kv8._E4M3, (kv8._E4M3[1:] + kv8._E4M3[:-1]) / 2,
                        np.array([448.0001, 2.0 ** -10, 2.0 ** -11, 3 * 2.0 ** -10, 0.0, -0.0])]).astype(np.float32)
    ref = torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(kv8.e4m3_codes(y), ref)
    codes = np.arange(256, dtype=np.uint8)
    ref = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(kv8.code_values(codes, "e4m3"), ref, equal_nan=True)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_code_is_within_half_a_step_of_the_value(kind):
    """|x - code scale| <= half a step of the code grid, but for the roundings of scale and 1 / scale: in exact
    rationals over every pair of bf16 significands and many exponents, RN32(x RN32(1 / scale)) is off x / scale by
    at most 3 * 2^-24 relative, so the code is a nearest one of a value that close."""
    rng = np.random.default_rng(0)
    for ma in range(128, 256, 7):
        a = ma / 128.0
        mx = rng.integers(128, 256, 64)
        x = mx / 128.0 * 2.0 ** -rng.integers(0, 12, 64)
        x = np.where(x <= a, x, a) * rng.choice([-1, 1], 64)
        codes, scale = kv8.quantise(np.concatenate([[a], x])[None, :], kind)
        c = kv8.code_values(codes, kind)[0, 1:]
        for xi, ci in zip(x, c):
            y = Fraction(float(xi)) / Fraction(float(scale))
            if kind == "int8":
                step = Fraction(1)
            else:
                e = max(-6, int(np.floor(np.log2(max(abs(float(y)), 2.0 ** -9)))))
                step = Fraction(2) ** (e - 3)
            assert abs(y - Fraction(float(ci))) <= step / 2 * (1 + Fraction(1, 8) * (kind == "e4m3")) + abs(y) * 3 * Fraction(1, 2 ** 24)
    assert np.abs(kv8.code_values(codes, kind)).max() == kv8.TOP[kind]


def test_scales_of_special_blocks():
    x = np.ones((3, 128))
    for bad in (np.nan, np.inf, -np.inf):
        y = x.copy()
        y[1, 5] = bad
        codes, scale = kv8.quantise(y, "int8")
        assert np.isnan(scale) and not codes.any()
    assert kv8.quantise(x * 2.0 ** -101, "e4m3")[1] == 0
    assert kv8.quantise(x * 0, "int8")[1] == 0
    codes, scale = kv8.quantise(x, "int8")
    assert scale == np.float32(1 / 127) and (codes == 127).all()


def test_values_held_are_near_the_rows():
    rows = bf16.from_f32((np.random.default_rng(1).standard_normal((130, 128)) * 3).astype(np.float32))
    x = bf16.to_f64(rows)
    for kind, rel in (("int8", 0.02), ("e4m3", 0.04)):
        h = kv8.held(rows, kind)
        assert h.shape == x.shape and np.linalg.norm(h - x) < rel * np.linalg.norm(x)


def test_attend_brute_force():
    rng = np.random.default_rng(2)
    q, K, V = rng.standard_normal((2, 128)), rng.standard_normal((5, 128)), rng.standard_normal((5, 128))
    out, w = kv8.attend(q, K, V, np.array([1, 4]))
    for i, n in ((0, 2), (1, 5)):
        c = [30 * np.tanh(float(np.dot(q[i], K[j])) / 128 ** 0.5 / 30) for j in range(n)]
        e = np.exp(c)
        assert np.allclose(out[i], sum(e[j] * V[j] for j in range(n)) / e.sum(), rtol=1e-12)
        assert np.allclose(w[i].sum(), 1) and not w[i, n:].any()


def test_block_weights_add_up():
    w = np.random.default_rng(3).random((6, 130))
    b = kv8.block_weights(w, 5)
    assert np.allclose(b[:3], [w[:, :64].sum(), w[:, 64:128].sum(), w[:, 128:].sum()]) and not b[3:].any()


def test_evict_by_hand():
    table, weight = list(range(10, 18)), [5.0, 1.0, 3.0, 3.0, np.nan, 2.0, 9.0, 7.0]
    # six full blocks and an open one; the first and the last full block stay, 3.0 at index 2 before 3.0 at 3
    t, w, n = kv8.evict(table, weight, 6 * 64 + 5, keep=3, sink=1, recent=1)
    assert t == [10, 12, 15, 16, 11, 13, 14, 17] and n == 3 * 64 + 5
    assert w == [5.0, 3.0, 2.0, 9.0, 0.0, 0.0, 0.0, 7.0]
    assert kv8.evict(table, weight, 3 * 64 + 5, 3, 0, 0)[0] == table
    assert kv8.evict(table, weight, 8 * 64, 1, 0, 0)[0] == [16, 10, 11, 12, 13, 14, 15, 17]
