"""Calls on quantised caches whose bounded waits are given next to no time: each
answer is right or reported, a warp's lanes give up together (what follows a
wait are warp-wide instructions), and the calls after it are right."""


import pytest
import torch

import sink_augmented_gqa_b200 as sa
from sink_augmented_gqa_b200 import workloads as wl

from helpers import check_bf16_output
from test_gpu_int4 import _setup

pytestmark = pytest.mark.gpu
DEV = "cuda"
DEFAULT_LIMIT = 2_000_000_000


@pytest.mark.parametrize("limit", [0, 300, 3000])
@pytest.mark.parametrize("fmt", ["int4", "fp8"])
@pytest.mark.parametrize("over,off", [(dict(B=40, n_q=16, n_kv=8, d=64), 700), (dict(B=2, n_q=8, n_kv=2, d=96), 3000),
                                      (dict(B=3, n_q=16, n_kv=2, d=128), 2500)])
def test_short_waits_are_right_or_reported(cuda_device, fmt, over, off, limit):
    T = 20
    cfg, cache, oracle, cos, sin = _setup(over, fmt, off, 2 * T)
    ws = sa.decode_workspace(cfg.B, cfg.n_q, cfg.n_kv, cfg.d, device=DEV)
    decode_in, prefill_in = wl.qkv(cfg, 1, step=1), wl.qkv(cfg, T, step=2)
    snap, osnap = cache.snapshot(), oracle.cache.snapshot()

    def calls():
        res = []
        for rows, name in ((decode_in, "decode"), (prefill_in, "prefill")):
            args = (cache, *(t.to(DEV) for t in rows), None, 0, cfg.sm_scale, cos, sin)
            if name == "decode":
                out = sa.attn_decode(*args, workspace=ws)
            else:
                out = sa.attn_prefill_quant(*args)
            torch.cuda.synchronize()
            res.append((name, out, sa.device_status()))
            cache.restore(snap)
        return res

    refs = {}
    for rows, name in ((decode_in, "decode"), (prefill_in, "prefill")):
        refs[name] = oracle.call(*rows, None, 0, read=fmt == "int4" or name == "prefill")[0]
        oracle.cache.restore(osnap)
    assert sa.device_status() == "SA_OK"
    sa.set_wait_limit(limit)
    try:
        short = calls()
    finally:
        sa.set_wait_limit(DEFAULT_LIMIT)
    print([(name, status) for name, _, status in short])
    for name, out, status in short:
        assert status in ("SA_OK", "SA_ERR_TIMEOUT"), (name, status)
        if status == "SA_OK":
            check_bf16_output(out, refs[name], f"{name} with a limit of {limit}")
    assert torch.count_nonzero(ws[: 8 * cfg.B * cfg.n_kv]) == 0   # tickets and stage counters
    for name, out, status in calls():
        assert status == "SA_OK"
        check_bf16_output(out, refs[name], f"{name} afterwards")
