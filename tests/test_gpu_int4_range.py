"""INT4 decode with block scales of V far apart, and with blocks of V that are
not finite: every block of 32 outputs is compared on its own scale, and the
lse, which knows nothing of V.

The bound of an output element, from the rounding steps that reach it
(alpha_j the weights, v_j the stored values, s_j the scale of their block):

* P' = alpha s in f16: half a step, 2^-11, of each alpha_j |v_j|. As much again
  covers the exponentials and fp32 sums: 2^-10 sum_j alpha_j |v_j| together.
* P' below f16's normal range: half of its last step, 2^-25, of 8 codes at most,
  in units of 2^(E - 6) <= 2^-2 max_j alpha_j s_j, for each of N keys, twice that
  where E trails a rising score by its rounding: N 2^-23 max_j alpha_j s_j.
* the tensor core's truncated sums, 136 2^-22 of alpha_j s_j at most over the two
  products of 16 keys: 2^-14 sum_j alpha_j s_j.
* the bf16 output: half a step.
"""

import math

import numpy as np
import pytest
import torch

import sink_augmented_gqa_b200 as sa
from oracle import int4 as oint4
from sink_augmented_gqa_b200 import workloads as wl

from helpers import check_lse, half_step, to64

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _attend(q, K, V, sink, scale):
    """One head in fp64: (out [d], bound [d], lse) of query q [d] over rows K, V [n, d]."""
    x = K @ q * scale
    m = max(x.max(), sink)
    w = np.exp(x - m)
    total = w.sum() + np.exp(sink - m)
    a = (w / total)[:, None]
    s = np.repeat(np.abs(oint4.quantize_rows(V)[1]), oint4.BLOCK, axis=-1)
    out = (a * V).sum(0)
    e = (2.0 ** -10 * (a * np.abs(V)).sum(0) + len(x) * 2.0 ** -23 * (a * s).max(0) + 2.0 ** -14 * (a * s).sum(0))
    return out, half_step(np.abs(out) + e) + e, m + np.log(total)


def _check(q, k, v, kn, vn, sinks, window=0, what="", static=False):
    """Decode row (kn, vn) [n_kv, d] and queries q [n_q, d] behind rows k, v
    [n, n_kv, d] (bf16, K as stored), and compare. Blocks of V that hold
    something not finite read as NaN, for every head that attends them."""
    n, n_kv, d = k.shape
    n_q = q.shape[0]
    sm = 1 / math.sqrt(d)
    cache = sa.KVCache(1, (n + 16) // 16 * 16, n_kv, d, device=DEV, int4=True)
    if n:
        cache.append(k[None].to(DEV), v[None].to(DEV))
    args = (cache, q[None, None].to(DEV), kn[None, None].to(DEV), vn[None, None].to(DEV),
            None if sinks is None else sinks.to(DEV), window, sm)
    out, lse = (sa.attn_decode_static if static else sa.attn_decode)(*args, rope_fused=False, return_lse=True)
    out, lse = to64(out)[0, 0], to64(lse)[0, :, 0]
    lo = max(0, n + 1 - window) if window else 0
    K = oint4.stored_rows(to64(torch.cat([k, kn[None]])[lo:]))
    V = oint4.stored_rows(to64(torch.cat([v, vn[None]])[lo:]))
    ref_lse = np.zeros(n_q)
    for h in range(n_q):
        g = h // (n_q // n_kv)
        bad = np.isnan(V[:, g]).any(0)
        ref, bound, ref_lse[h] = _attend(to64(q[h]), K[:, g], np.nan_to_num(V[:, g]),
                                         -np.inf if sinks is None else float(sinks[h]), sm)
        assert np.isnan(out[h][bad]).all(), f"{what}: head {h}: finite where the block is not"
        err = np.abs(out[h] - ref)[~bad]
        worst = (err / bound[~bad]).max() if err.size else 0.0
        assert np.all(err <= bound[~bad]), f"{what}: head {h}: error {worst} of its bound"
    check_lse(torch.from_numpy(lse), ref_lse, what)


def _rows(n, n_q, n_kv, d, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)   # noqa: E731
    return r(n_q, d), r(n, n_kv, d), r(n, n_kv, d), r(n_kv, d), r(n_kv, d), torch.randn(n_q, generator=g)


SHAPES = [(8, 1, 64), (6, 2, 96), (8, 2, 128)]


@pytest.mark.parametrize("n_q,n_kv,d", SHAPES)
@pytest.mark.parametrize("n", [40, 600, 2047])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_a_block_that_is_not_finite_stays_in_its_block(cuda_device, n_q, n_kv, d, n, value):
    for block in range(d // 32):
        q, k, v, kn, vn, sinks = _rows(n, n_q, n_kv, d, block)
        v[n * (block + 1) // (d // 32 + 1), n_kv - 1, 32 * block + 5] = value
        _check(q, k, v, kn, vn, sinks, what=f"{value} in block {block}")


@pytest.mark.parametrize("n_q,n_kv,d", SHAPES)
def test_the_new_row_is_not_finite_in_a_block(cuda_device, n_q, n_kv, d):
    q, k, v, kn, vn, sinks = _rows(300, n_q, n_kv, d)
    vn[0, d - 1] = math.nan
    _check(q, k, v, kn, vn, sinks, what="new row")
    _check(q, k, v, kn, vn, sinks, window=100, what="new row, band")
    _check(q, k[:0], v[:0], kn, vn, None, what="new row alone")


@pytest.mark.parametrize("n_q,n_kv,d", SHAPES)
@pytest.mark.parametrize("power", [1, 10, 18, 25, 40, 60, 90, -10, -40, -90])
def test_blocks_far_apart(cuda_device, n_q, n_kv, d, power):
    for block in (0, d // 32 - 1):
        q, k, v, kn, vn, sinks = _rows(1500, n_q, n_kv, d, power)
        v[..., 32 * block:32 * block + 32] *= 2.0 ** power
        vn[..., 32 * block:32 * block + 32] *= 2.0 ** power
        _check(q, k, v, kn, vn, sinks, what=f"block {block} times 2^{power}")
        _check(q, k, v, kn, vn, sinks, window=200, what=f"block {block} times 2^{power}, band", static=True)


@pytest.mark.parametrize("n_q,n_kv,d", SHAPES)
@pytest.mark.parametrize("power", [10, 18, 25, 40, 60])
def test_rows_far_apart(cuda_device, n_q, n_kv, d, power):
    q, k, v, kn, vn, sinks = _rows(1500, n_q, n_kv, d, power)
    for blk in range(d // 32):   # one element of one row in each block, at a place of its own
        v[97 + 411 * blk % 1400, 0, 32 * blk + 3] = 2.0 ** power
    _check(q, k, v, kn, vn, sinks, what=f"elements of 2^{power}")
    v[::7] *= 2.0 ** -power
    _check(q, k, v, kn, vn, sinks, what=f"elements of 2^{power}, rows of 2^-{power}")


@pytest.mark.parametrize("n_q,n_kv,d", SHAPES)
@pytest.mark.parametrize("size", [1e3, 1e8, 1e10, 1e20])
@pytest.mark.parametrize("at", [0, 33, 900, 2047])
def test_a_huge_row_without_weight(cuda_device, n_q, n_kv, d, size, at):
    # its score lies 40 nats (2^-58) under the others': all heads of a group look one way
    n = 2048
    q, k, v, kn, vn, sinks = _rows(n, n_q, n_kv, d)
    m = n_q // n_kv
    k *= 0.25
    for g in range(n_kv):
        base = q[g * m].float()
        q[g * m:(g + 1) * m] = (base * torch.linspace(0.9, 1.1, m)[:, None]).to(torch.bfloat16)
        k[at, g] = (-40.0 * math.sqrt(d) / base.square().sum() * base).to(torch.bfloat16)
    v[..., 0] = 4.0
    vn[..., 0] = 4.0
    v[at] *= size
    _check(q, k, v, kn, vn, sinks, what=f"{size} at {at}")


@pytest.mark.parametrize("n_q,n_kv,d", SHAPES)
def test_a_huge_row_that_one_head_of_a_group_attends(cuda_device, n_q, n_kv, d):
    n, at = 1000, 555
    q, k, v, kn, vn, sinks = _rows(n, n_q, n_kv, d)
    m = n_q // n_kv
    k *= 0.25
    for g in range(n_kv):
        base = q[g * m].float()
        sign = torch.tensor([1.0 if i % 2 else -1.0 for i in range(m)])
        q[g * m:(g + 1) * m] = (base * sign[:, None]).to(torch.bfloat16)
        k[at, g] = (-40.0 * math.sqrt(d) / base.square().sum() * base).to(torch.bfloat16)
    v[at] *= 1e9
    _check(q, k, v, kn, vn, sinks, what="one head's huge row")


@pytest.mark.parametrize("n_q,n_kv,d", SHAPES)
@pytest.mark.parametrize("nats", [45.0, -45.0])
def test_scores_rise_as_values_fall(cuda_device, n_q, n_kv, d, nats):
    # scores rise (or fall) by 65 powers of two over the rows and values go the
    # other way, so that every row counts alike: ref and E move all along
    n = 3000
    q, k, v, kn, vn, _ = _rows(n, n_q, n_kv, d)
    m = n_q // n_kv
    t = torch.linspace(0.0, nats, n)
    for g in range(n_kv):
        base = q[g * m].float()
        q[g * m:(g + 1) * m] = base.to(torch.bfloat16)
        k[:, g] = (t[:, None] * math.sqrt(d) / base.square().sum() * base).to(torch.bfloat16)
    v = (v.float() * torch.exp(-t)[:, None, None]).to(torch.bfloat16)
    _check(q, k, v, kn, vn, None, what="falling values")


@pytest.mark.parametrize("over,n", [(dict(B=1, n_q=8, n_kv=1, d=64), 5000), (dict(B=30, n_q=16, n_kv=8, d=64), 700),
                                    (dict(B=3, n_q=16, n_kv=2, d=128), 3000)])
def test_identical_calls_give_identical_bits(cuda_device, over, n):
    cfg = wl.scaled(wl.CONFIGS["tiny"], **over)
    cache = sa.KVCache(cfg.B, (n + 16) // 16 * 16, cfg.n_kv, cfg.d, device=DEV, int4=True)
    cache.append(*(t.to(DEV) for t in wl.prefilled_cache_rows(cfg, rows=n)))
    q, k, v = (t.to(DEV) for t in wl.qkv(cfg, 1, step=1))
    ws = sa.decode_workspace(cfg.B, cfg.n_q, cfg.n_kv, cfg.d, device=DEV)
    snap, first = cache.snapshot(), None
    for _ in range(20):
        cache.restore(snap)
        got = sa.attn_decode(cache, q, k, v, None, 0, cfg.sm_scale, rope_fused=False, workspace=ws, return_lse=True)
        first = first or got
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])
