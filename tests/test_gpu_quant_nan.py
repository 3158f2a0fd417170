"""Prefill, on caches of every format, with a key that is not a number: every query row
that attends it is NaN, its lse too, wherever in a tile the key lies (some of a
tile's exponentials are a polynomial, some the hardware's), and the rows whose
mask leaves it out are as without it."""

import math

import numpy as np
import pytest
import torch

import sink_augmented_gqa_b200 as sa
from sink_augmented_gqa_b200 import workloads as wl

from helpers import check_bf16_output, check_lse
from test_gpu_int4 import _append, _cache, _setup

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("fmt", ["int4", "fp8", "bf16"])
@pytest.mark.parametrize("over,off,T,window", [
    (dict(B=1, n_q=8, n_kv=2, d=64), 200, 150, 0),      # whole query tiles
    (dict(B=1, n_q=8, n_kv=2, d=64), 200, 150, 128),    # a band, heads packed
    (dict(B=1, n_q=8, n_kv=4, d=96), 200, 150, 128),    # a band, whole query tiles
    (dict(B=1, n_q=5, n_kv=1, d=128), 3000, 6, 0),      # few rows behind many: parts
    (dict(B=2, n_q=16, n_kv=2, d=64), 4000, 3, 0)],
    ids=["full", "band", "band96", "parts128", "parts64"])
def test_a_key_that_is_not_a_number(cuda_device, fmt, over, off, T, window):
    cfg, cache, oracle, cos, sin = _setup(over, fmt, off, T)
    q, k, v = wl.qkv(cfg, T, step=1)
    sinks = wl.sinks(cfg)
    ref, ref_lse, _ = oracle.call(q, k, v, sinks, window)
    kp, vp = wl.prefilled_cache_rows(cfg, rows=off)
    for j in [off - 1 - i for i in range(8)] + [off + min(i, T - 1) for i in range(0, 8, 3)]:
        kj, kn = kp.clone(), k.clone()
        (kj[:, j] if j < off else kn[:, j - off])[:, 0, 7] = math.nan
        cache = _cache(fmt, cfg.B, (off + T + 15) // 16 * 16, cfg.n_kv, cfg.d)
        _append(cache, kj, vp)
        prefill = sa.attn_prefill if fmt == "bf16" else sa.attn_prefill_quant
        out, lse = prefill(cache, q.to(DEV), kn.to(DEV), v.to(DEV), sinks.to(DEV), window, cfg.sm_scale, cos, sin,
                           return_lse=True)
        pos = off + np.arange(T)
        sees = (pos >= j) & ((window == 0) | (pos - j < window))
        m = cfg.n_q // cfg.n_kv                           # the heads of KV head 0
        assert torch.isnan(out[:, torch.from_numpy(sees), :m]).all(), f"key {j}: a row that attends it is finite"
        assert torch.isnan(lse[:, :m, torch.from_numpy(sees)]).all(), f"key {j}: a finite lse"
        check_bf16_output(out[:, torch.from_numpy(~sees)], ref[:, ~sees], f"key {j}: rows that mask it")
        check_lse(lse[:, :, torch.from_numpy(~sees)], ref_lse[:, :, ~sees], f"key {j}: lse of rows that mask it")
        if cfg.n_kv > 1:
            check_bf16_output(out[:, :, m:], ref[:, :, m:], f"key {j}: the other heads")
            check_lse(lse[:, m:], ref_lse[:, m:], f"key {j}: lse of the other heads")
