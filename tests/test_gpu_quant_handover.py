"""Rows read back from a quantised cache, appended to a bf16 one and decoded
there: the answer is the oracle's over the rows as they read back, for both
formats, full layers and bands."""

import numpy as np
import pytest
import torch

import sink_augmented_gqa_b200 as sa
from sink_augmented_gqa_b200 import workloads as wl

from helpers import check_bf16_output, check_lse, to64
from test_gpu_int4 import _setup

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("fmt", ["int4", "fp8"])
@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("window", [0, 128], ids=["full", "band"])
def test_gone_on_with_in_bf16(cuda_device, fmt, d, window):
    cfg, cache, oracle, cos, sin = _setup(dict(B=2, n_q=16, n_kv=2, d=d), fmt, 150, 50, ring_window=window)
    sinks = wl.sinks(cfg)
    q, k, v = wl.qkv(cfg, 40, step=1)
    out = sa.attn_prefill_quant(cache, q.to(DEV), k.to(DEV), v.to(DEV), sinks.to(DEV), window, cfg.sm_scale, cos, sin)
    check_bf16_output(out, oracle.call(q, k, v, sinks, window)[0], f"{fmt} turn")
    n = cache.offset
    kb, vb = cache.read(0, n)
    assert np.array_equal(to64(kb), oracle.cache.K[:, :n]) and np.array_equal(to64(vb), oracle.cache.V[:, :n])
    plain = sa.KVCache(cfg.B, n + 16, cfg.n_kv, cfg.d, device=DEV)
    plain.append(kb, vb)
    oracle.fmt = "bf16"                      # the bf16 cache's new rows are not quantised
    for step in range(2):
        q, k, v = wl.qkv(cfg, 1, step=40 + step)
        out, lse = sa.attn_decode(plain, q.to(DEV), k.to(DEV), v.to(DEV), sinks.to(DEV), window, cfg.sm_scale, cos, sin,
                                  return_lse=True)
        torch.cuda.synchronize()
        ref, ref_lse, _ = oracle.call(q, k, v, sinks, window)
        check_bf16_output(out, ref, f"{fmt} rows in bf16, step {step}")
        check_lse(lse, ref_lse, f"{fmt} rows in bf16, step {step}")
