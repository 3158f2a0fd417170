"""4-bit KV-cache rows with one bf16 scale per 32 elements: quantise, dequantise.

TEST INFRASTRUCTURE (see ``oracle/__init__.py``).

The MoE-Xtend README lists quantisation-aware long-context runs, with KV and
its dequantisation first because decode is bandwidth bound ("ROADMAP"). The
codes are those of the published Q4_0 scheme (the ``u`` below over blocks of
32 with ``s = -m / 8``); the scale's 5 bits, the tie of ``m`` and ``-m``, zeros
and NaNs are this library's own:

* blocks of 32 consecutive elements of a bf16 row; ``m`` is the block's element
  of largest magnitude (the positive one where ``m`` and ``-m`` both occur);
* ``s = -m / 8`` rounded to 5 significant bits (nearest, ties to even);
* ``u = min(15, floor(x / s + 8.5))``, one of 0..15 (``m`` itself gets 0);
* a reader sees ``s * (u - 8)``: at most 5 + 3 significant bits, so exactly a
  bf16 number;
* a block with ``|m| < 2**-120`` is all zeros (``s = 0``, ``u = 8``), a block
  with an infinity or a NaN all NaN (``s`` NaN, ``u = 8``).

Two codes share a byte, the even element in the low half.
"""

import numpy as np

BLOCK = 32
SMALLEST = 2.0 ** -120


def _blocks(x):
    return x.reshape(x.shape[:-1] + (x.shape[-1] // BLOCK, BLOCK))


def quantize_rows(x):
    """Quantise the last axis (a multiple of 32) of bf16-representable fp64
    ``x``. Returns ``(codes uint8 0..15, x's shape; scales fp64 [..., d/32])``.
    The division is exact enough in fp64: ``x / s`` is a border between codes
    only where the quotient is representable."""
    b = _blocks(np.asarray(x, dtype=np.float64))
    with np.errstate(invalid="ignore", over="ignore"):
        bad = ~np.isfinite(b).all(axis=-1)
        c = np.where(np.isfinite(b), b, 0.0)
        hi, lo = c.max(axis=-1), c.min(axis=-1)
        m = np.where(hi >= -lo, hi, lo)
        frac, exp = np.frexp(-m / 8)
        s = np.where(np.abs(m) < SMALLEST, 0.0, np.ldexp(np.rint(frac * 32), exp - 5))
        y = c / np.where(s == 0, 1.0, s)[..., None]
        u = np.clip(np.floor(y + 8.5), 0, 15)
    u = np.where((bad | (s == 0))[..., None], 8, u).astype(np.uint8)
    s = np.where(bad, np.nan, s)
    return u.reshape(np.shape(x)), s


def dequantize_rows(codes, scales):
    """fp64 values a reader of the quantised cache sees."""
    return (_blocks(codes.astype(np.float64) - 8) * scales[..., None]).reshape(codes.shape)


def pack(codes):
    """uint8 bytes [..., d/2] of codes [..., d]."""
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(packed):
    out = np.empty(packed.shape[:-1] + (2 * packed.shape[-1],), dtype=np.uint8)
    out[..., 0::2], out[..., 1::2] = packed & 15, packed >> 4
    return out


def stored_rows(x):
    """What the rows ``x`` stand for once they are in the cache."""
    return dequantize_rows(*quantize_rows(x))


def kv_bytes_int4(L, B, T, H_kv, d):
    """The "KV CACHE" estimator with half a byte per element and a bf16 scale
    per 32 elements, K and V."""
    return 2 * L * B * T * H_kv * (d // 2 + 2 * d // BLOCK)
