"""The INT4 row format: the oracle against brute force and closed forms (CPU)."""

import os
import re

import numpy as np
import pytest

from sink_augmented_gqa_b200 import fit_exp2_poly as F
from oracle import bf16 as obf16
from oracle import int4 as oint4


def _rows(n, d, seed, scale=1.0):
    return obf16.round_bf16(np.random.default_rng(seed).standard_normal((n, d)) * scale)


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("scale", [1.0, 1e-20, 3e30])
def test_codes_are_nearest_and_errors_bounded(d, scale):
    x = _rows(400, d, 1, scale)
    u, s = oint4.quantize_rows(x)
    assert u.min() >= 0 and u.max() <= 15 and s.shape == (400, d // 32)
    back = oint4.dequantize_rows(u, s)
    # brute force: no other code of the block's scale is nearer
    levels = (np.arange(16) - 8.0) * s[..., None]
    b = x.reshape(400, d // 32, 32)
    best = np.abs(levels[:, :, None, :] - b[..., None]).min(axis=-1)
    err = np.abs(back - x).reshape(b.shape)
    assert np.array_equal(err, best)
    m = np.abs(b).max(axis=-1, keepdims=True)
    assert (err <= m / 6).all()
    sign = np.where(b.max(axis=-1, keepdims=True) == m, 1.0, -1.0)   # of the block's m
    unclipped = (np.abs(b) <= 7 / 8 * m) | (np.sign(b) == sign)
    assert (err[unclipped] <= np.broadcast_to(m / 15, b.shape)[unclipped]).all()


def test_stored_values_are_bf16_numbers_and_requantise_to_themselves():
    x = np.concatenate([_rows(300, 64, 2), _rows(300, 64, 3, 1e-30), _rows(300, 64, 4, 1e30)])
    u, s = oint4.quantize_rows(x)
    back = oint4.dequantize_rows(u, s)
    assert np.array_equal(obf16.round_bf16(back), back)
    assert np.array_equal(obf16.round_bf16(s), s)
    u2, s2 = oint4.quantize_rows(back)
    assert np.array_equal(s, s2) and np.array_equal(oint4.dequantize_rows(u2, s2), back)
    # the same codes, but for a tie of m and -8 s: a block cannot hold +8 steps
    assert np.array_equal(u, u2)


def test_scale_and_code_by_hand():
    x = np.zeros((1, 32))
    x[0, :6] = [-4.0, 4.0, 0.25, -0.25, 0.24, 3.75]
    u, s = oint4.quantize_rows(x)
    assert s[0, 0] == -0.5                       # the positive one of the tie leads
    # 4 / -0.5 = -8 -> 0; -4 -> 8, clipped to 15; 0.25 / -0.5 = -0.5, a border, goes up to 8;
    # -0.25 -> 0.5 goes up to 9; 0.24 -> 8; 3.75 -> -7.5 goes up to 1
    assert u[0, :7].tolist() == [15, 0, 8, 9, 8, 1, 8]


def test_scale_rounds_to_five_significant_bits():
    x = np.zeros((2, 32))
    x[0, 3], x[1, 3] = -8 * (1 + 9 / 128), 8 * (1 + 12 / 128)
    _, s = oint4.quantize_rows(x)
    assert s[0, 0] == 1 + 1 / 16                 # 1.0703 is nearer to 1.0625 than to 1.125
    assert s[1, 0] == -(1 + 2 / 16)              # 1.09375, a tie of 1.0625 and 1.125: the even one


def test_zero_tiny_and_nonfinite_blocks():
    x = np.zeros((5, 64))
    x[1, 5] = 2.0 ** -120
    x[2, 5] = -(2.0 ** -121)
    x[3, 40], x[3, 1] = np.inf, 1.0
    x[4, 2] = np.nan
    u, s = oint4.quantize_rows(x)
    back = oint4.dequantize_rows(u, s)
    assert (back[0] == 0).all() and (u[0] == 8).all() and (s[0] == 0).all()
    assert back[1, 5] == 2.0 ** -120 and (back[2] == 0).all()
    assert np.isnan(back[3, 32:]).all() and back[3, 1] == 1.0 and np.isfinite(back[3, :32]).all()
    assert np.isnan(back[4, :32]).all() and (back[4, 32:] == 0).all()


def test_packing_and_bytes():
    u = np.random.default_rng(5).integers(0, 16, (3, 96)).astype(np.uint8)
    p = oint4.pack(u)
    assert p.shape == (3, 48) and p[0, 0] == u[0, 0] + 16 * u[0, 1]
    assert np.array_equal(oint4.unpack(p), u)
    # 24 layers, 131,072 positions, 8 heads of 64: 6.0 GiB in bf16 (2 bytes an element) at 4.5 bits
    assert oint4.kv_bytes_int4(24, 1, 131072, 8, 64) * 16 == 6 * 2 ** 30 * 4.5


def test_fine_exp2_coefficients():
    """The degree-4 polynomial of the prefill on quantised caches is what the
    fit gives, within 3.5e-6 in fp32 Horner form."""
    text = open(os.path.join(os.path.dirname(F.__file__), "csrc", "ptx.cuh")).read()
    c = np.array([float(v) for _, v in sorted(re.findall(r"EXP2F_C(\d) = ([0-9.e+-]+)f", text))], dtype=np.float32)
    np.testing.assert_allclose(c, F.fit(4), rtol=2e-6)
    assert F.max_rel_error(c) < 3.5e-6


def test_reciprocal_form_of_the_codes():
    """The kernel's arithmetic, sat(fma(x, 1/(15 s), (8 + 2^-11) / 15)) times 15
    rounded to the nearest integer, equals min(15, floor(x/s + 8.5)) for every
    pair of significands, with a reciprocal a few steps off."""
    f = np.float32
    wrong = 0
    for M in range(128, 256):
        m = M / 16.0
        frac, exp = np.frexp(-m / 8)
        s = np.ldexp(np.rint(frac * 32), exp - 5)
        xs = np.concatenate([np.arange(128, 256) * 2.0 ** k for k in range(-24, 1)])
        xs = xs[xs / 16 <= m] / 16
        xs = np.concatenate([xs, -xs, [0.0]])
        want = np.minimum(15, np.floor(xs / s + 8.5))
        for steps in (-2, 0, 2):
            r = f(f(1 / 15) / f(s))
            for _ in range(abs(steps)):
                r = np.nextafter(r, f(np.sign(steps) * 1e30))
            y = np.clip((xs * np.float64(r) + np.float64(f((8 + 2.0 ** -11) / 15))).astype(f), 0, 1)
            wrong += int((np.rint((np.float64(y) * 15).astype(f)) != want).sum())
    assert wrong == 0
